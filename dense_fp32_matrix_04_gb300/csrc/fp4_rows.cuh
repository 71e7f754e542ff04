// The product of 4-bit operands for one token: the time is that of reading B, its
// codes and scales, once.
//
// A warp takes two rows of B at a time, 512 contiguous bytes of codes of each a load.
// Codes become FP16 numbers, two an instruction, and are multiplied with the token's
// codes, which are FP16 in shared memory (read once for both rows: read for each, they
// took longer than B), in packed FMAs: eight products of at most 36, in quarters, in each
// half, are exact (288 is 1152 quarters, below the 2048 that FP16 counts to).  The blocks'
// sums are then scaled and added in FP32.
//
// The scales of B lie in tiles of 128 rows by 4 blocks, where 32 bytes hold a word each of
// the rows 2 i, 2 i + 1 and those 32, 64 and 96 further on: four warps of a block take these
// pairs, so that what one reads of them serves all.  A token that comes unquantised is
// quantised by every block itself while its first rows of B are on their way.
//
// 4096 x 4096 takes 6.3 us with the token's quantisation and 5.7 without, with weights in turn (from
// HBM, 1.6 TB/s; the same weights in L2: 5.2 and 4.8): a launch, the token and one round of loads
// behind it.
#pragma once

#include <cuda_fp8.h>

#include <cstdint>

#include "fp4_mma.cuh"
#include "fp4_quantize.cuh"
#include "rows.cuh"

namespace sgemm {

constexpr int kFp4RowsThreads = 256;
constexpr int kFp4RowsPieces = 4;    // loads of 16 bytes a lane has in flight
constexpr int kFp4RowsChunk = 1024;  // columns of a warp's load
constexpr int kFp4RowsSmem = 200 * 1024;

// Columns of the token in shared memory: whole loads.
__host__ __device__ constexpr int64_t fp4_rows_columns(int K) { return ((int64_t)K + kFp4RowsChunk - 1) / kFp4RowsChunk * kFp4RowsChunk; }
// Its bytes: FP16 codes, an FP32 scale for every 16 columns (blocks of 32: two factors of one).
__host__ __device__ constexpr int64_t fp4_rows_smem(int K) { return fp4_rows_columns(K) / 16 * 36; }

// Place of columns c .. c + 7 (c a multiple of 8) among the token's codes: within a chunk, the four
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

// The power of two of an e8m0 scale as two factors of about its root: the product of two scales may
// leave FP32 where what they scale does not, that of two factors never does.
__device__ __forceinline__ float2 e8m0_factors(uint32_t s) {
    const int e = (int)s - 127, half = e >> 1;
    return make_float2(__uint_as_float((uint32_t)(127 + half) << 23),
                       __uint_as_float(s == 255 ? 0x7fc00000u : (uint32_t)(127 + e - half) << 23));
}
// What 32 columns are scaled by: two e4m3 scales of 16 columns each, or the factors of one e8m0.
template <int BLOCK>
__device__ __forceinline__ float2 fp4_scale_values(uint32_t s) {
    if constexpr (BLOCK == 16) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)s, __NV_E4M3);
        return __half22float2(__half2(h));
    } else {
        return e8m0_factors(s & 255u);
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
    int64_t ldb;
    const void *X;  // the token, where it is not quantised yet
};

// XT: the token is codes (-1) or values of that element type.
template <int XT, int BLOCK>
__global__ void __launch_bounds__(kFp4RowsThreads, 3) fp4_rows_kernel(const Fp4RowsArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ float slots[kFp4RowsThreads / 32];
    constexpr int WARPS = kFp4RowsThreads / 32;
    static_assert(WARPS == 8);
    const Fp4Args &p = a.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, K = p.K;
    const int columns = (int)fp4_rows_columns(K), n_tiles = fp4_tiles(K, BLOCK);
    __half *codes = reinterpret_cast<__half *>(smem);
    float *scales = reinterpret_cast<float *>(codes + columns);
    // a group is 16 rows, pairs 2 i and 2 i + 2 of 128 and the three that share their scales' sectors
    const int groups = (p.N + 127) / 128 * 8;
    int group = blockIdx.x;
    auto row_of = [&](int g) { return g / 8 * 128 + g % 8 * 4 + (warp >> 2) * 2 + (warp & 3) * 32; };

    uint4 w[2][kFp4RowsPieces];
    uint32_t ws[2][kFp4RowsPieces];
    auto load = [&](int row, int c0) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int j = 0; j < kFp4RowsPieces; ++j) {
                const int c = c0 + kFp4RowsChunk * j + 32 * lane;
                const bool in = row + r < p.N && c < K;
                // (rows are whole 16-byte pieces; what lies behind K meets a token of 0)
                w[r][j] = in ? __ldg(reinterpret_cast<const uint4 *>(a.B + (row + r) * a.ldb + c / 2)) : make_uint4(0, 0, 0, 0);
                ws[r][j] = in ? fp4_load_scales<BLOCK>(p.b_tiles, row + r, c / 32, n_tiles) : 0u;
            }
    };
    int row = row_of(group);
    load(row, 0);

    auto put = [&](int c, const __half2 (&h)[4]) {
        *reinterpret_cast<uint4 *>(codes + fp4_rows_place(c)) = *reinterpret_cast<const uint4 *>(h);
    };
    float row_scale = 1.f;
    if constexpr (XT < 0) {
        const int bytes = (K + 1) / 2;
        for (int c = 32 * tid; c < columns; c += 32 * kFp4RowsThreads) {
            const bool in = c < K;
            const uint4 q = in ? __ldg(reinterpret_cast<const uint4 *>(a.A + c / 2)) : make_uint4(0, 0, 0, 0);
            const uint32_t word[4] = {q.x, q.y, q.z, q.w};
            *reinterpret_cast<float2 *>(scales + c / 16) =
                fp4_scale_values<BLOCK>(in ? fp4_load_scales<BLOCK>(p.a_tiles, 0, c / 32, n_tiles) : 0u);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // bytes behind the row's end may hold anything
                const int left = bytes - c / 2 - 4 * i;
                __half2 h[4];
                e2m1x8_to_f16(left >= 4 ? word[i] : left > 0 ? word[i] & ((1u << 8 * left) - 1) : 0u, h);
                put(c + 8 * i, h);
            }
        }
        if (p.a_scale) row_scale = *p.a_scale;
    } else {
        // a thread takes 16 columns at a time
        constexpr int DT = XT < 0 ? 0 : XT;
        const typename Elem<DT>::type *x = static_cast<const typename Elem<DT>::type *>(a.X);
        Fp4Piece<DT, false> piece;
        F2 v[8];
        uint32_t top = 0, most = 0;
        if constexpr (BLOCK == 16) {
            // (the columns that the loop below begins with come last, and stay)
            for (int c = 16 * tid + (columns - 1) / (16 * kFp4RowsThreads) * (16 * kFp4RowsThreads); c >= 0; c -= 16 * kFp4RowsThreads) {
                piece.load(x, c, K);
                top = piece.unpack(x, c, K, v);
                most = max(most, top);
            }
            most = warp_max(most);
            if (lane == 0) slots[warp] = __uint_as_float(most);
            __syncthreads();
            for (int i = 0; i < WARPS; ++i) most = max(most, __float_as_uint(slots[i]));
        }
        const Fp4Row r(most);
        for (int c = 16 * tid; c < columns; c += 16 * kFp4RowsThreads) {
            if (BLOCK == 32 || c >= 16 * kFp4RowsThreads) {
                piece.load(x, c, K);
                top = piece.unpack(x, c, K, v);
            }
            uint2 q;
            const uint32_t s = fp4_encode<BLOCK>(v, top, r, q);
            __half2 h[4];
            e2m1x8_to_f16(q.x, h);
            put(c, h);
            e2m1x8_to_f16(q.y, h);
            put(c + 8, h);
            const float2 f = fp4_scale_values<BLOCK>(s);
            scales[c / 16] = BLOCK == 32 && (c & 16) ? f.y : f.x;
        }
        if (BLOCK == 16) row_scale = r.scale();
    }
    __syncthreads();

    for (; group < groups; group += gridDim.x) {
        float acc[2] = {0.f, 0.f};
        for (int c0 = 0; c0 < columns; c0 += kFp4RowsChunk * kFp4RowsPieces) {
            if (c0 > 0) load(row, c0);
#pragma unroll
            for (int j = 0; j < kFp4RowsPieces; ++j) {
                const int c = c0 + kFp4RowsChunk * j;
                if (c >= columns) break;
                const float2 sx = *reinterpret_cast<const float2 *>(scales + c / 16 + 2 * lane);
                __half2 s[2][2] = {};  // of each row, a half of the 32 columns each
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint4 q = *reinterpret_cast<const uint4 *>(codes + c + 8 * lane + i * 256);
                    const __half2 *x = reinterpret_cast<const __half2 *>(&q);
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const uint32_t word = i == 0 ? w[r][j].x : i == 1 ? w[r][j].y : i == 2 ? w[r][j].z : w[r][j].w;
                        __half2 b[4];
                        e2m1x8_to_f16(word, b);
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[r][i / 2] = __hfma2(b[e], x[e], s[r][i / 2]);
                    }
                }
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float2 sb = fp4_scale_values<BLOCK>(ws[r][j]), f = __half22float2(s[r][0]), g = __half22float2(s[r][1]);
                    if constexpr (BLOCK == 16) {
                        acc[r] = fmaf(f.x + f.y, sb.x * sx.x, acc[r]);
                        acc[r] = fmaf(g.x + g.y, sb.y * sx.y, acc[r]);
                    } else {
                        // (exact up to the last addition, and infinite only where the product is)
                        acc[r] = fmaf((f.x + f.y + g.x + g.y) * (sb.x * sx.x), sb.y * sx.y, acc[r]);
                    }
                }
            }
        }
        const int done = row + lane;
        row = row_of(group + gridDim.x);
        if (group + (int)gridDim.x < groups) load(row, 0);
        const float sums[2] = {warp_sum(acc[0]), warp_sum(acc[1])};
        if (lane < 2 && done < p.N)
            store_c(p.C, done, p.ctype,
                    fmaf((lane ? sums[1] : sums[0]) * row_scale, p.b_scale ? p.b_scale[done] : 1.f, p.bias ? p.bias[done] : 0.f));
    }
}

}  // namespace sgemm
