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
//
// 8192 x 8192 BF16 takes 35 us in blocks of 16 and 28 in blocks of 32 (172 MB, 4.9 and 6.1
// TB/s), FP32 52 and 46: instructions and memory in equal parts, some 14 a warp for 32
// elements, and in blocks of 16 the row's maximum, a barrier, before any code is known.
// Odd rows are shifted: 30000 x 1001 FP32 35 us, 3.9 TB/s.  Rows of more than 16384 columns are read
// twice in blocks of 16: 1024 x 32768 BF16 28 us, in blocks of 32 17.5 (86 MB).
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
__device__ __forceinline__ uint32_t e2m1x8(const F2 *v) {
    const float2 a = v[0].both(), b = v[1].both(), c = v[2].both(), d = v[3].both();
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}\n"
        : "=r"(r)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y), "f"(d.x), "f"(d.y));
    return r;
}

// A row's factor 2688 / max and its scale, from the bits of the largest magnitude
// in it (a NaN counts as the largest).  Below 2^-100 the quotient could overflow:
// such rows are first multiplied by 2^64, exactly.  Rows that are not finite have
// factor 0, so codes of 0, and a scale that is not finite.
struct Fp4Row {
    float pre = 1.f, t = 0.f, m;
    __device__ float scale() const { return __fdiv_rn(m, 2688.f); }
    __device__ explicit Fp4Row(uint32_t max_bits) {
        m = __uint_as_float(max_bits);
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
__device__ __forceinline__ uint32_t fp4_encode(F2 (&v)[8], uint32_t top, const Fp4Row &r, uint2 &codes) {
    uint32_t s;
    float inv;
    if constexpr (BLOCK == 16) {
        if (r.pre != 1.f)  // (few rows)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = v[i] * F2(r.pre);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] * F2(r.t);
        // of products with one factor the largest is the product of the largest
        s = fp4_scale16(r.t > 0.f ? __uint_as_float(top) * r.pre * r.t : 0.f, inv);
    } else {
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        s = fp4_scale32(top, inv);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] * F2(inv);
    codes = make_uint2(e2m1x8(v), e2m1x8(v + 4));
    if (inv == 0.f) codes = make_uint2(0, 0);
    return s;
}

// The codes and the scale of columns c .. c + 15 of row m are written; as fp4_encode, with the
// first lane's c a multiple of 512.
template <int BLOCK>
__device__ __forceinline__ void fp4_put(const Fp4Rows &a, int64_t m, int c, F2 (&v)[8], uint32_t top, const Fp4Row &r) {
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
    // four scales to a word, which the first of its threads has; those of blocks behind the row are 0
    constexpr int EACH = BLOCK / 16, LANES = 4 * EACH;  // threads a scale, a word
    if (!in) s = 0;
    s |= __shfl_down_sync(0xffffffffu, s, EACH) << 8;
    s |= __shfl_down_sync(0xffffffffu, s, 2 * EACH) << 16;
    const int n_tiles = fp4_tiles(a.K, BLOCK), tile = c / (16 * LANES);
    if (threadIdx.x % LANES == 0 && tile < n_tiles) *reinterpret_cast<uint32_t *>(a.tiles + fp4_scale_word(m, tile, n_tiles)) = s;
}

// The larger magnitude of two numbers, or of two pairs of 16-bit ones.
template <int DT>
__device__ __forceinline__ uint32_t max_magnitude(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (DT == SGEMM_F32) asm("max.NaN.xorsign.abs.f32 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
    else if constexpr (DT == SGEMM_BF16) asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
    else asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// 16 columns of a row from column c (a multiple of 16) on.  ALIGNED: the row starts on 16 bytes and
// consists of whole pieces of 16 bytes; any other row is read as the pieces that enclose it, of which
// nothing behind the one with its last byte, and shifted.
template <int DT, bool ALIGNED>
struct Fp4Piece {
    using type = typename Elem<DT>::type;
    static constexpr int VEC = Elem<DT>::VEC, N = 16 / VEC, PIECES = N + (ALIGNED ? 0 : 1);
    uint4 raw[PIECES];
    // A warp's pieces, its first lane's column c0 on, into shared memory, beside each other as they lie
    // in the row (sectors that two instructions read half of each would be read twice); and a lane's
    // from there.
    static constexpr int WARP_PIECES = 32 * N + (ALIGNED ? 0 : 1);
    __device__ static void copy(uint4 *slot, int lane, const type *row, int c0, int K) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(row + c0) & ~(uintptr_t)15, end = c0 < K ? reinterpret_cast<uintptr_t>(row + K) : 0;
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int p = 32 * i + lane;
            if (i < N || lane == 0)
                cp_async_16(smem_addr(slot + p), reinterpret_cast<const void *>(at + 16 * p), at + 16 * p < end ? 16 : 0);
        }
    }
    __device__ void take(const uint4 *slot, int lane) {
#pragma unroll
        for (int i = 0; i < PIECES; ++i) raw[i] = slot[N * lane + i];
    }
    __device__ void load(const type *row, int c, int K) {
        if constexpr (ALIGNED) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                raw[i] = c + i * VEC < K ? __ldg(reinterpret_cast<const uint4 *>(row + c + i * VEC)) : make_uint4(0, 0, 0, 0);
        } else {
            const uintptr_t at = reinterpret_cast<uintptr_t>(row + c) & ~(uintptr_t)15, end = reinterpret_cast<uintptr_t>(row + K);
#pragma unroll
            for (int i = 0; i <= N; ++i)
                raw[i] = c < K && at + 16 * i < end ? __ldg(reinterpret_cast<const uint4 *>(at + 16 * i)) : make_uint4(0, 0, 0, 0);
        }
    }
    // the values, 0 from column K on, and the bits of the largest magnitude among them
    __device__ uint32_t unpack(const type *row, int c, int K, F2 (&v)[8]) const {
        uint4 w[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if constexpr (ALIGNED) w[i] = raw[i];
            else w[i] = shift_bytes(raw[i], raw[i + 1], (unsigned)(reinterpret_cast<uintptr_t>(row) & 15));
        }
        if (!ALIGNED && c + 16 > K) {
            uint32_t *words = reinterpret_cast<uint32_t *>(w);
#pragma unroll
            for (int i = 0; i < 4 * N; ++i) {
                const int left = K - c - i * VEC / 4;  // elements from the word's first on
                if constexpr (DT == SGEMM_F32) words[i] = left > 0 ? words[i] : 0u;
                else words[i] = left > 1 ? words[i] : left > 0 ? words[i] & 0xffffu : 0u;
            }
        }
        // magnitudes, a NaN before all: one instruction for two operands (signs come out wrong, and go)
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            top = max_magnitude<DT>(max_magnitude<DT>(top, max_magnitude<DT>(w[i].x, w[i].y)), max_magnitude<DT>(w[i].z, w[i].w));
            float x[VEC];
            unpack16<DT>(w[i], x);
#pragma unroll
            for (int e = 0; e < VEC / 2; ++e) v[i * VEC / 2 + e] = F2(x[2 * e], x[2 * e + 1]);
        }
        if constexpr (DT == SGEMM_F32) {
            top &= 0x7fffffffu;
        } else {
            // (bits of magnitudes order as the magnitudes do)
            const uint32_t half = max(top & 0x7fffu, top >> 16 & 0x7fffu);
            if constexpr (DT == SGEMM_BF16) top = half << 16;
            else top = __float_as_uint(__half2float(__ushort_as_half((unsigned short)half)));
        }
        return top;
    }
};

// A row to the threads of blockDim.x, EACH times 16 columns a thread; blocks walk several rows: the next
// is on its way into each warp's own places in shared memory while one is worked on (into registers:
// 8192 x 8192 BF16 39.5 us, so 32.9; with three rows on their way fewer blocks fit, 35.4 and FP32 76.9
// instead of 51.5).
constexpr int kFp4RowSlots = 2;
template <int DT, bool ALIGNED, int BLOCK, int EACH>
__global__ void __launch_bounds__(EACH == 1 ? 256 : 512)
    quantize_fp4_kernel(const Fp4Rows a, const typename Elem<DT>::type *__restrict__ x, int64_t ldx) {
    using Piece16 = Fp4Piece<DT, ALIGNED>;
    constexpr int SLOT = Piece16::WARP_PIECES, DEPTH = kFp4RowSlots;
    extern __shared__ __align__(16) uint4 ring[];
    __shared__ float slots[RowReducer::SLOTS];
    griddep_launch_dependents();
    RowReducer red{slots, (int)(blockDim.x >> 5)};
    const int c0 = threadIdx.x * 16, across = blockDim.x * 16, step = gridDim.x * blockDim.y;
    const int lane = threadIdx.x & 31, warp = (threadIdx.y * blockDim.x + threadIdx.x) >> 5;
    uint4 *mine = ring + warp * DEPTH * EACH * SLOT;
    auto copy = [&](int64_t m, int stage) {
        if (m < a.M)
#pragma unroll
            for (int g = 0; g < EACH; ++g)
                Piece16::copy(mine + (stage * EACH + g) * SLOT, lane, x + m * ldx, c0 + g * across - 16 * lane, a.K);
        cp_async_commit();
    };
    const int64_t first = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
#pragma unroll
    for (int s = 0; s < DEPTH - 1; ++s) copy(first + (int64_t)s * step, s);
    int stage = 0;
    for (int64_t m = first; m < a.rows; m += step) {
        F2 v[EACH][8];
        uint32_t top[EACH], most = 0;
        cp_async_wait<DEPTH - 2>();
        __syncwarp();
#pragma unroll
        for (int g = 0; g < EACH; ++g) {
            Piece16 piece;
            piece.take(mine + (stage * EACH + g) * SLOT, lane);
            top[g] = piece.unpack(x + m * ldx, c0 + g * across, m < a.M ? a.K : 0, v[g]);
            most = max(most, top[g]);
        }
        copy(m + (int64_t)(DEPTH - 1) * step, stage == 0 ? DEPTH - 1 : stage - 1);
        stage = stage == DEPTH - 1 ? 0 : stage + 1;
        const Fp4Row r(BLOCK == 16 ? red.max(most) : 0u);
        if (BLOCK == 16 && threadIdx.x == 0 && m < a.M) a.scale[m] = r.scale();
#pragma unroll
        for (int g = 0; g < EACH; ++g) fp4_put<BLOCK>(a, m, c0 + g * across, v[g], top[g], r);
    }
}

// Rows wider than the registers of a block: read a second time where the row's
// largest is needed first.
template <int DT, bool ALIGNED, int BLOCK>
__global__ void __launch_bounds__(1024)
    quantize_fp4_wide_kernel(const Fp4Rows a, const typename Elem<DT>::type *__restrict__ x, int64_t ldx) {
    __shared__ float slots[RowReducer::SLOTS];
    griddep_launch_dependents();
    RowReducer red{slots, (int)(blockDim.x >> 5)};
    const int step = blockDim.x * 16, first = threadIdx.x * 16, end = (a.K + 511) / 512 * 512;
    Fp4Piece<DT, ALIGNED> piece;
    F2 v[8];
    for (int64_t m = blockIdx.x; m < a.rows; m += gridDim.x) {
        uint32_t top = 0;
        if (BLOCK == 16 && m < a.M)
            for (int c = first; c < a.K; c += step) {
                piece.load(x + m * ldx, c, a.K);
                top = max(top, piece.unpack(x + m * ldx, c, a.K, v));
            }
        const Fp4Row r(BLOCK == 16 ? red.max(top) : 0u);
        if (BLOCK == 16 && threadIdx.x == 0 && m < a.M) a.scale[m] = r.scale();
        for (int c = first; c < end; c += step) {
            piece.load(x + m * ldx, c, m < a.M ? a.K : 0);
            top = piece.unpack(x + m * ldx, c, m < a.M ? a.K : 0, v);
            fp4_put<BLOCK>(a, m, c, v, top, r);
        }
    }
}

// Scales from rows of plain bytes to tiles; those outside the matrix are 0.  For weights, once: byte by
// byte, 8192 x 512 8.7 us, 1 TB/s.
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
