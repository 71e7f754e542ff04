// Rows quantised to 4-bit floating point (e2m1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and
// their negatives) with a scale for each block of 16 or 32 columns.
//
// Blocks of 16: the row is first scaled to a largest magnitude of 2688 = 448 * 6,
// y = x (2688 / max|row|), so that the blocks' scales s = e4m3(max|y| / 6) use the
// whole of their range, up to 448; the codes are e2m1(y (1 / s)), and the row's own
// scale, max|row| / 2688, is FP32.  Blocks of 32: s is the smallest power of two with
// max|x| / s <= 6 (e8m0), the codes are e2m1(x / s), and there is no row scale.
// Every operation is an FP32 one rounded once, so codes and scales are defined to
// the bit.
//
// A thread takes 16 columns: 8 bytes of codes, and a scale, or half of one.  The
// scales go to where the tensor cores want them, tiles of 128 rows by 4 blocks.
#pragma once

#include <cuda_fp8.h>

#include <cstdint>

#include "ptx.cuh"
#include "rows.cuh"

namespace sgemm {

// Tiles of 128 rows by 4 blocks: byte 16 (r % 32) + 4 (r / 32 % 4) + j % 4 of the
// 512 of tile (r / 128, j / 4) is the scale of row r and block j; a row of tiles is
// contiguous.
constexpr int kFp4TileBytes = 512;
__host__ __device__ constexpr int fp4_blocks(int K, int block) { return (K - 1) / block + 1; }
__host__ __device__ constexpr int fp4_tiles(int K, int block) { return (fp4_blocks(K, block) + 3) / 4; }
__host__ __device__ inline int64_t fp4_scale_word(int64_t row, int tile, int tiles) {
    return ((row >> 7) * tiles + tile) * kFp4TileBytes + (row & 31) * 16 + ((row >> 5) & 3) * 4;
}

// Eight FP32 values as codes, the first in the lowest four bits.
__device__ __forceinline__ uint32_t e2m1x8(const float *v) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}\n"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// A row's factor 2688 / max and its scale, from the bits of the largest magnitude
// in it (a NaN counts as the largest).  Below 2^-100 the quotient could overflow:
// such rows are first multiplied by 2^64, exactly.  Rows that are not finite have
// factor 0, so codes of 0, and a scale that is not finite.
struct Fp4Row {
    float pre = 1.f, t = 0.f, scale;
    __device__ explicit Fp4Row(uint32_t max_bits) {
        const float m = __uint_as_float(max_bits);
        scale = __fdiv_rn(m, 2688.f);
        if (max_bits > 0 && max_bits < 0x7f800000u) {
            if (m < 0x1p-100f) pre = 0x1p64f;
            t = __fdiv_rn(2688.f, m * pre);
        }
    }
};

// The scale of a block of 16 as e4m3 bits, and what its (scaled) columns are
// multiplied with, from their largest magnitude.
__device__ __forceinline__ uint32_t fp4_scale16(float top, float &inv) {
    const uint32_t s = __nv_cvt_float_to_fp8(__fmul_rn(top, 1.f / 6.f), __NV_SATFINITE, __NV_E4M3);
    const float v = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)s, __NV_E4M3)));
    inv = s ? __frcp_rn(v) : 0.f;
    return s;
}

// The same of a block of 32 as e8m0 bits: the exponent of the largest magnitude
// less two, one more where its fraction is above 1.5; NaN (255) for blocks that are
// not finite.
__device__ __forceinline__ uint32_t fp4_scale32(uint32_t max_bits, float &inv) {
    if (max_bits >= 0x7f800000u) {
        inv = 0.f;
        return 255u;
    }
    const int e = max((int)(max_bits >> 23) - 2 + ((max_bits & 0x7fffffu) > 0x400000u), 0);
    inv = __uint_as_float((uint32_t)(254 - e) << 23);
    return (uint32_t)e;
}

// Where the codes and the scales go.
struct Fp4Rows {
    int M, rows, K;  // rows from M up to `rows` have scales of 0 and no codes
    uint8_t *q;
    int64_t ldq;
    uint8_t *tiles;
    float *scale;
};

// The codes of 16 columns, from their values and their largest magnitude's bits, and the bits
// of their block's scale; all lanes of a warp call it, neighbours with columns beside each other.
template <int BLOCK>
__device__ __forceinline__ uint32_t fp4_encode(float (&v)[16], uint32_t top, const Fp4Row &r, uint2 &codes) {
    uint32_t s;
    float inv;
    if constexpr (BLOCK == 16) {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = v[i] * r.pre * r.t;
        // of products with one factor the largest is the product of the largest
        s = fp4_scale16(r.t > 0.f ? __uint_as_float(top) * r.pre * r.t : 0.f, inv);
    } else {
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        s = fp4_scale32(top, inv);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] *= inv;
    codes = make_uint2(e2m1x8(v), e2m1x8(v + 8));
    if (inv == 0.f) codes = make_uint2(0, 0);
    return s;
}

// The codes and the scale of columns c .. c + 15 of row m are written; as fp4_encode, with the
// first lane's c a multiple of 512.
template <int BLOCK>
__device__ __forceinline__ void fp4_put(const Fp4Rows &a, int64_t m, int c, float (&v)[16], uint32_t top, const Fp4Row &r) {
    uint2 codes;
    uint32_t s = fp4_encode<BLOCK>(v, top, r, codes);
    const bool in = m < a.M && c < a.K;
    if (in) {
        uint8_t *to = a.q + m * a.ldq + c / 2;
        const int left = (a.K + 1) / 2 - c / 2;
        if (left >= 8) {
            *reinterpret_cast<uint2 *>(to) = codes;
        } else {
            for (int i = 0; i < left; ++i) to[i] = (uint8_t)((i < 4 ? codes.x : codes.y) >> (8 * (i & 3)));
        }
    }
    // four scales to a word; those of blocks behind the row are 0
    constexpr int EACH = BLOCK / 16, LANES = 4 * EACH;  // threads a scale, a word
    if (!in) s = 0;
    const int lane = threadIdx.x & 31, n_tiles = fp4_tiles(a.K, BLOCK), tile = c / (16 * LANES);
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) word |= __shfl_sync(0xffffffffu, s, (lane & ~(LANES - 1)) + i * EACH) << (8 * i);
    if (lane % LANES == 0 && tile < n_tiles) *reinterpret_cast<uint32_t *>(a.tiles + fp4_scale_word(m, tile, n_tiles)) = word;
}

// 16 columns of a row from column c on, in 16-byte pieces (VW) or by single elements (VW 1).
template <int DT, int VW>
struct Fp4Piece {
    using P = Piece<DT, VW>;
    static constexpr int N = 16 / VW;
    typename P::raw raw[N];
    __device__ void load(const typename P::type *row, int c, int K) {
#pragma unroll
        for (int i = 0; i < N; ++i) raw[i] = c + i * VW < K ? P::load(row + c + i * VW) : P::zero();
    }
    // the values, and the bits of the largest magnitude among them
    __device__ uint32_t unpack(float (&v)[16]) const {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) P::unpack(raw[i], v + i * VW);
#pragma unroll
        for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
        return top;
    }
};

// A row to the threads of blockDim.x, once; blocks walk several rows.
template <int DT, int VW, int BLOCK>
__global__ void __launch_bounds__(1024)
    quantize_fp4_kernel(const Fp4Rows a, const typename Elem<DT>::type *__restrict__ x, int64_t ldx) {
    __shared__ float slots[RowReducer::SLOTS];
    griddep_launch_dependents();
    RowReducer red{slots, (int)(blockDim.x >> 5)};
    const int c = threadIdx.x * 16, step = gridDim.x * blockDim.y;
    Fp4Piece<DT, VW> next;
    auto load = [&](int64_t m) { next.load(x + m * ldx, c, m < a.M ? a.K : 0); };
    constexpr bool AHEAD = VW == 8;  // the next row is on its way while this one is reduced and written
    if (AHEAD) load((int64_t)blockIdx.x * blockDim.y + threadIdx.y);
    for (int64_t m = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; m < a.rows; m += step) {
        float v[16];
        if (!AHEAD) load(m);
        const uint32_t top = next.unpack(v);
        if (AHEAD) load(m + step);
        const Fp4Row r(BLOCK == 16 ? red.max(top) : 0u);
        if (BLOCK == 16 && threadIdx.x == 0 && m < a.M) a.scale[m] = r.scale;
        fp4_put<BLOCK>(a, m, c, v, top, r);
    }
}

// Rows wider than the registers of a block: read a second time where the row's
// largest is needed first.
template <int DT, int VW, int BLOCK>
__global__ void __launch_bounds__(1024)
    quantize_fp4_wide_kernel(const Fp4Rows a, const typename Elem<DT>::type *__restrict__ x, int64_t ldx) {
    __shared__ float slots[RowReducer::SLOTS];
    griddep_launch_dependents();
    RowReducer red{slots, (int)(blockDim.x >> 5)};
    const int step = blockDim.x * 16, first = threadIdx.x * 16, end = (a.K + 511) / 512 * 512;
    Fp4Piece<DT, VW> piece;
    float v[16];
    for (int64_t m = blockIdx.x; m < a.rows; m += gridDim.x) {
        uint32_t top = 0;
        if (BLOCK == 16 && m < a.M)
            for (int c = first; c < a.K; c += step) {
                piece.load(x + m * ldx, c, a.K);
                top = max(top, piece.unpack(v));
            }
        const Fp4Row r(BLOCK == 16 ? red.max(top) : 0u);
        if (BLOCK == 16 && threadIdx.x == 0 && m < a.M) a.scale[m] = r.scale;
        for (int c = first; c < end; c += step) {
            piece.load(x + m * ldx, c, m < a.M ? a.K : 0);
            top = piece.unpack(v);
            fp4_put<BLOCK>(a, m, c, v, top, r);
        }
    }
}

// Scales from rows of plain bytes to tiles; those outside the matrix are 0.
__global__ void __launch_bounds__(256)
    fp4_lay_out_scales_kernel(int rows, int blocks, const uint8_t *__restrict__ s, int64_t lds, uint8_t *__restrict__ tiles) {
    const int n_tiles = (blocks + 3) / 4;
    const int64_t words = ((int64_t)rows + 127) / 128 * 128 * n_tiles;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < words; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t row = i / n_tiles;
        const int tile = (int)(i - row * n_tiles);
        uint32_t word = 0;
        for (int j = 0; j < 4; ++j)
            if (row < rows && 4 * tile + j < blocks) word |= (uint32_t)s[row * lds + 4 * tile + j] << (8 * j);
        *reinterpret_cast<uint32_t *>(tiles + fp4_scale_word(row, tile, n_tiles)) = word;
    }
}

}  // namespace sgemm
