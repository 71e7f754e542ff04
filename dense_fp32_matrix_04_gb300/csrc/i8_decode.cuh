// The product of 8-bit operands for few rows of A (up to 64, the tokens of a
// decoding step): the time is that of reading B, N K bytes, once.
//
// B goes from memory to registers, 16 bytes a thread and load, and becomes the
// A fragments of mma.sync.m16n8k16 there: the sum over k may be taken in any
// order, so the four FP16 pairs that a thread holds for a k-step are 4
// consecutive bytes of a row instead of two pairs eight apart, and the tokens'
// fragments are read with the same order from shared memory, where their codes
// lie as FP16.  Each block takes 16 R rows of B; its eight warps share k, and
// the blocks of a cluster share k again where there are few rows of B.  The
// loads of B are issued before the tokens are waited for.
#pragma once

#include <cstdint>

#include "i8_codes.cuh"
#include "ptx.cuh"

namespace sgemm {

__device__ __forceinline__ void mma_f16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// R tiles of 16 rows of B, NT tiles of 8 tokens, BPW blocks of 64 k a warp
// between two rounds of staging tokens.
template <int R_, int NT_, int BPW_>
struct I8DecodeTile {
    static constexpr int R = R_, NT = NT_, BPW = BPW_, WARPS = 8, THREADS = 256;
    static constexpr int ROWS = 16 * R, TOKENS = 8 * NT, KC = WARPS * BPW * 64;
    // a token's codes: the 16 bytes of padding keep the fragments' reads free of bank conflicts
    static constexpr int PITCH = KC * 2 + 16;
    static constexpr int SUMS = WARPS * ROWS * TOKENS * 4;
    static constexpr int STAGE = TOKENS * PITCH;
    static constexpr int SMEM = (STAGE > SUMS ? STAGE : SUMS) + ROWS * TOKENS * 4;
};

template <class T, bool ALIGNED_A, bool ALIGNED_B>
__global__ void __launch_bounds__(T::THREADS, T::NT < 8 ? 2 : 1) i8_decode_kernel(const I8Args p, int ranks) {
    constexpr int R = T::R, NT = T::NT, BPW = T::BPW;
    extern __shared__ __align__(16) unsigned char smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    const int rank = blockIdx.x % ranks, row0 = (int)(blockIdx.x / ranks) * T::ROWS;
    const int blocks = (p.K + 63) / 64;
    const int k_begin = (int)((int64_t)blocks * rank / ranks) * 64, k_end = (int)((int64_t)blocks * (rank + 1) / ranks) * 64;

    const int8_t *b_row[2 * R];
#pragma unroll
    for (int i = 0; i < 2 * R; ++i) b_row[i] = p.B + min((int64_t)row0 + 8 * i + g, (int64_t)p.N - 1) * p.ldb;

    float acc[R][NT][4];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[r][n][i] = 0.f;

    for (int kc = k_begin; kc < k_end; kc += T::KC) {
        uint4 w[BPW][2 * R];
#pragma unroll
        for (int j = 0; j < BPW; ++j) {
            const int k = kc + (warp * BPW + j) * 64 + 16 * t4;
#pragma unroll
            for (int i = 0; i < 2 * R; ++i)
                w[j][i] = k < k_end ? load_codes<ALIGNED_B>(b_row[i], k, p.K) : make_uint4(0, 0, 0, 0);
        }
        if (kc == k_begin) griddep_wait();  // the tokens may come from the kernel before
        else __syncthreads();               // the tokens of the round before have been read
        const int pieces = min(T::KC, k_end - kc + 15) / 16;
        for (int i = tid; i < T::TOKENS * (T::KC / 16); i += T::THREADS) {
            const int n = i / (T::KC / 16), piece = i % (T::KC / 16), k = kc + piece * 16;
            if (piece >= pieces) continue;
            uint4 c = make_uint4(0, 0, 0, 0);
            if (n < p.M && k < p.K) {
                c = load_codes<ALIGNED_A>(p.A + n * p.lda, k, p.K);
                if (k + 16 > p.K) {
                    // nothing past the row's end: what B holds there is multiplied by 0
                    uint32_t v[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int left = p.K - k - 4 * e;
                        v[e] = left <= 0 ? 0u : left >= 4 ? v[e] : v[e] & ((1u << (8 * left)) - 1u);
                    }
                    c = make_uint4(v[0], v[1], v[2], v[3]);
                }
            }
            const uint2 c0 = i8x4_to_f16(c.x), c1 = i8x4_to_f16(c.y), c2 = i8x4_to_f16(c.z), c3 = i8x4_to_f16(c.w);
            uint4 *to = reinterpret_cast<uint4 *>(smem + n * T::PITCH + piece * 32);
            to[0] = make_uint4(c0.x, c0.y, c1.x, c1.y);
            to[1] = make_uint4(c2.x, c2.y, c3.x, c3.y);
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < BPW; ++j) {
            const int kb = (warp * BPW + j) * 64;
            if (kc + kb >= k_end) break;
            uint2 a[2 * R][4];
#pragma unroll
            for (int i = 0; i < 2 * R; ++i) {
                a[i][0] = i8x4_to_f16(w[j][i].x);
                a[i][1] = i8x4_to_f16(w[j][i].y);
                a[i][2] = i8x4_to_f16(w[j][i].z);
                a[i][3] = i8x4_to_f16(w[j][i].w);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint4 *x = reinterpret_cast<const uint4 *>(smem + (8 * n + g) * T::PITCH + kb * 2 + t4 * 32);
                const uint4 x0 = x[0], x1 = x[1];
                const uint32_t b[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
#pragma unroll
                for (int s = 0; s < 4; ++s)
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        mma_f16_16816(acc[r][n], a[2 * r][s].x, a[2 * r + 1][s].x, a[2 * r][s].y, a[2 * r + 1][s].y,
                                      b[2 * s], b[2 * s + 1]);
            }
        }
    }
    if (k_begin >= k_end) griddep_wait();

    // add the warps' sums, then the ranks', each in order
    __syncthreads();
    float *sums = reinterpret_cast<float *>(smem);
    float *block_sums = reinterpret_cast<float *>(smem + T::SMEM - T::ROWS * T::TOKENS * 4);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                sums[(warp * T::TOKENS + 8 * n + 2 * t4 + (i & 1)) * T::ROWS + 16 * r + g + 8 * (i >> 1)] = acc[r][n][i];
    __syncthreads();
    constexpr int OUTPUTS = T::ROWS * T::TOKENS;
    const int used = T::ROWS * min(T::TOKENS, p.M);
    auto output = [&](int i, float s) {
        const int m = i / T::ROWS, n = row0 + i % T::ROWS;
        if (n < p.N) {
            s *= p.a_scale[m];
            store_c(p.C, m * p.ldc + n, p.ctype, fmaf(s, p.b_scale[n], p.bias ? p.bias[n] : 0.f));
        }
    };
    for (int i = tid; i < used; i += T::THREADS) {
        float s = sums[i];
#pragma unroll
        for (int w = 1; w < T::WARPS; ++w) s += sums[w * OUTPUTS + i];
        if (ranks == 1) output(i, s);
        else block_sums[i] = s;
    }
    if (ranks > 1) {
        __syncwarp();
        cluster_sync();
        for (int i = tid * ranks + rank; i < used; i += T::THREADS * ranks) {
            float s = 0.f;
            for (int r = 0; r < ranks; ++r)
                s += __uint_as_float(dsmem_ld_u32(dsmem_map(smem_addr(block_sums + i), (uint32_t)r)));
            output(i, s);
        }
        __syncwarp();
        cluster_sync();
    }
}

}  // namespace sgemm
