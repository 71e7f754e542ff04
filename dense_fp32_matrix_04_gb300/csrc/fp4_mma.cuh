// The product of 4-bit operands with block scales on the 5th-generation tensor
// cores: tcgen05.mma multiplies the codes, scales the products of each block and
// adds them up in FP32; the rows' scales and the bias follow when the accumulator
// is drained.
//
// A tile is 128 rows of B, the weights, by up to 256 tokens, transposed: lanes of
// tensor memory are rows of B, columns tokens.  A k-step is 256 columns, 128 bytes
// of codes a row, which TMA copies into swizzled rows; the scales, already laid out
// in tiles of 512 bytes (fp4_quantize.cuh), follow as plain bulk copies and go on
// into tensor memory by tcgen05.cp, issued in front of the products that use them.
//
// One block per SM walks tiles: one thread copies into a ring, one issues, four
// warps drain.  Where there are few tiles, a cluster of blocks shares each: every
// block adds up a part of K and the parts are joined through distributed shared
// memory, in a fixed order.  Every wait is bounded; a block that gives up records an
// error code and frees its tensor memory.
#pragma once

#include <cuda.h>

#include <cstdint>

#include "fp4_quantize.cuh"
#include "ptx.cuh"
#include "tcgen05.cuh"
#include "tile_map.cuh"

namespace sgemm {

struct Fp4Args {
    int M, N, K;
    const uint8_t *a_tiles, *b_tiles;  // block scales of the tokens and of B
    const float *a_scale, *b_scale, *bias;  // any may be null: 1, 1, 0
    void *C;
    int64_t ldc;
    int ctype;
};

// D[tmem] (+)= A[smem desc] * B[smem desc]^T over 64 columns of e2m1 codes, with
// scales in tensor memory: e4m3 for blocks of 16, e8m0 for blocks of 32.
template <int BLOCK>
__device__ __forceinline__ void umma_fp4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t a_scale, uint32_t b_scale, uint32_t accumulate) {
    if constexpr (BLOCK == 16)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(
                d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(a_scale), "r"(b_scale), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(
                d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(a_scale), "r"(b_scale), "r"(accumulate)
            : "memory");
}

// 512 bytes of scales, 32 rows of 16 bytes, into four columns of tensor memory, the
// same in each quarter of its lanes; in order with the products issued after it.
__device__ __forceinline__ void tmem_copy_scales(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n" ::"r"(taddr), "l"(desc) : "memory");
}
// Descriptor of such 512 bytes: rows of 16 bytes, 8 of them every 128 bytes, not swizzled.
__device__ __forceinline__ uint64_t umma_desc_scales(uint32_t saddr) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1u << 46);
}

// `bytes` (a multiple of 16) from global to shared memory, both 16-byte aligned.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

template <int TOK_, int BLOCK_>
struct Fp4Tile {
    static constexpr int ROWS = 128, TOK = TOK_, BLOCK = BLOCK_;
    static constexpr int BK = 256, BYTES = BK / 2;  // a k-step's columns, and bytes of codes a row
    static constexpr int DRAIN = 2, THREADS = 32 * (DRAIN + 4);
    // 512-byte tiles of scales: along a k-step, and of the 128 rows each that the tokens reach into.
    // A product's scales start on an even column of tensor memory, 64 rows: narrower tiles serve only
    // where one holds all tokens.
    static constexpr int KT = BK / BLOCK / 4, XT = TOK <= 128 ? 1 : 2;
    static constexpr int W_BYTES = ROWS * BYTES, X_BYTES = TOK * BYTES;
    static constexpr int WS_BYTES = KT * kFp4TileBytes, XS_BYTES = XT * WS_BYTES;
    static constexpr int STAGE = W_BYTES + X_BYTES + WS_BYTES + XS_BYTES;
    static constexpr int STAGES_FIT = (227 * 1024 - 1024 - 256) / STAGE, STAGES = STAGES_FIT > 8 ? 8 : STAGES_FIT;
    static constexpr int SMEM_BYTES = STAGES * STAGE + 1024 + 256;
    // tensor memory: accumulators, then two places for the scales of a k-step
    static constexpr int ACCS = TOK <= 192 ? 2 : 1, ACC_COLS = TOK < 32 ? 32 : TOK;
    static constexpr int SCALES = ACCS * ACC_COLS, SCALE_COLS = 4 * KT * (1 + XT), TMEM_COLS = 512;
    // A = B = e2m1 (1 at bits 7 and 10), both K-major, N >> 3 at bit 17, e8m0 scales at bit 23, M >> 4 at
    // bit 24; which pair of bytes of a scale's word is used, at bits 4 (B) and 29 (A)
    static constexpr uint32_t IDESC = (1u << 7) | (1u << 10) | ((uint32_t)(TOK >> 3) << 17) |
                                      ((BLOCK == 32 ? 1u : 0u) << 23) | ((uint32_t)(ROWS >> 4) << 24);
    static constexpr uint32_t SECOND_PAIR = (2u << 4) | (2u << 29);
    static_assert(TOK == 16 || TOK == 32 || TOK == 64 || (TOK % 64 == 0 && TOK <= 256), "columns of one product");
    static_assert(STAGES >= 4 && SCALES + 2 * SCALE_COLS <= TMEM_COLS, "a ring, and tensor memory");
};

// Unit u is tile u / splits, part u % splits of K (the rank in the cluster); with
// splits > 1 a block has one unit.  Tiles run over the tokens first within groups of
// eight tiles of rows, so that blocks at work together share both operands in L2.
// debug: the test-only switches (bit 0: no copies, so that the waits run out).
template <int TOK, int BLOCK>
__global__ void __launch_bounds__(Fp4Tile<TOK, BLOCK>::THREADS, 1)
    fp4_mma_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const Fp4Args p,
                   int splits, int *__restrict__ err_word, unsigned long long wait_limit_ns, int debug) {
    using T = Fp4Tile<TOK, BLOCK>;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    unsigned char *smem = smem_raw + (base - raw);
    // stages of the tokens, of B (128-byte swizzled boxes start on 1024 bytes), of their scales; the barriers
    const uint32_t w_base = base + T::STAGES * T::X_BYTES, ws_base = w_base + T::STAGES * T::W_BYTES;
    const uint32_t xs_base = ws_base + T::STAGES * T::WS_BYTES, bars = xs_base + T::STAGES * T::XS_BYTES;
    // copies done, stage read by the products; accumulator final, accumulator read
    const uint32_t full0 = bars, empty0 = full0 + 8 * T::STAGES;
    const uint32_t acc_full0 = empty0 + 8 * T::STAGES, acc_empty0 = acc_full0 + 8 * T::ACCS;
    const uint32_t drained = acc_empty0 + 8 * T::ACCS;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + (drained + 8 - base));
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + (drained + 12 - base));

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int tiles_n = (p.N + T::ROWS - 1) / T::ROWS, tiles_m = (p.M + TOK - 1) / TOK;
    const int units = tiles_m * tiles_n * splits;
    const int steps = (p.K + T::BK - 1) / T::BK, k_tiles = fp4_tiles(p.K, BLOCK), m_tiles = (p.M + 127) / 128;
    auto unit = [&](int u, int &m0, int &n0, int &k0, int &n) {
        int tn, tm;
        grouped_tile<8>(u / splits, tiles_n, tiles_m, tn, tm);
        m0 = tm * TOK;
        n0 = tn * T::ROWS;
        const int s = u % splits;
        k0 = (int)((int64_t)steps * s / splits);
        n = (int)((int64_t)steps * (s + 1) / splits) - k0;
    };

    if (warp == 0) {
        tmem_alloc(smem_addr(tmem_slot), T::TMEM_COLS);
        tmem_relinquish();
    }
    if (tid == 32) {
        for (int s = 0; s < T::STAGES; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int b = 0; b < T::ACCS; ++b) {
            mbar_init(acc_full0 + 8 * b, 1);
            mbar_init(acc_empty0 + 8 * b, 4);  // one arrival per drain warp
        }
        mbar_init(drained, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;

    int issued = 0;  // copies: k-steps issued over all of this block's units
    if (warp == 0) {
        RingPlace<T::STAGES> s;
        if (lane == 0) {
            prefetch_tensor_map(&tmW);
            prefetch_tensor_map(&tmX);
        }
        // Copies of step k of a unit into a stage: B's part, which announces both, and the tokens'.
        auto copy_b = [&](uint32_t at, int k, int m0, int n0) {
            if (elect_one()) {
                const uint32_t kt = (uint32_t)min(T::KT, k_tiles - k * T::KT) * kFp4TileBytes;
                const uint32_t xt = (uint32_t)min(T::XT, m_tiles - m0 / 128);
                mbar_arrive_expect_tx(full0 + 8 * at, T::W_BYTES + T::X_BYTES + kt * (1 + xt));
                tma_load_2d(w_base + at * T::W_BYTES, &tmW, k * T::BYTES, n0, full0 + 8 * at);
                bulk_load(ws_base + at * T::WS_BYTES, p.b_tiles + ((int64_t)(n0 / 128) * k_tiles + k * T::KT) * kFp4TileBytes,
                          kt, full0 + 8 * at);
            }
        };
        auto copy_tokens = [&](uint32_t at, int k, int m0) {
            if (elect_one()) {
                const uint32_t kt = (uint32_t)min(T::KT, k_tiles - k * T::KT) * kFp4TileBytes;
                tma_load_2d(base + at * T::X_BYTES, &tmX, k * T::BYTES, m0, full0 + 8 * at);
#pragma unroll
                for (int r = 0; r < T::XT; ++r)
                    if (m0 / 128 + r < m_tiles)
                        bulk_load(xs_base + at * T::XS_BYTES + r * T::WS_BYTES,
                                  p.a_tiles + ((int64_t)(m0 / 128 + r) * k_tiles + k * T::KT) * kFp4TileBytes, kt, full0 + 8 * at);
            }
        };
        // The tokens' codes may come from the kernel before; B does not: the first unit's first stages
        // of it are on their way before that kernel is waited for.
        int ahead = 0, m0, n0, k0, n;
        if (!(debug & 1) && (int)blockIdx.x < units) {
            unit(blockIdx.x, m0, n0, k0, n);
            for (ahead = min(n, T::STAGES); issued < ahead; ++issued) copy_b(issued, k0 + issued, m0, n0);
        }
        griddep_wait();
        for (int k = 0; k < ahead; ++k, s.next()) copy_tokens(k, k0 + k, m0);
        bool ok = true;
        for (int u = blockIdx.x; ok && !(debug & 1) && u < units; u += gridDim.x) {
            unit(u, m0, n0, k0, n);
            for (int k = k0 + (u == (int)blockIdx.x ? ahead : 0); k < k0 + n; ++k) {
                if (issued >= T::STAGES) ok = mbar_wait_polite(empty0 + 8 * s.at, s.round ^ 1, wait_limit_ns, 0);
                if (!__all_sync(0xffffffffu, ok)) {
                    *abort_flag = 1;
                    ok = false;
                    break;
                }
                copy_b(s.at, k, m0, n0);
                copy_tokens(s.at, k, m0);
                __syncwarp();
                ++issued;
                s.next();
            }
        }
    } else if (warp == 1) {
        // the whole warp walks the steps, so that addresses stay uniform; one lane issues
        RingPlace<T::STAGES> s, before;
        RingPlace<T::ACCS> b;
        const uint64_t x_desc0 = umma_desc_128b(base), w_desc0 = umma_desc_128b(w_base);
        const uint64_t xs_desc0 = umma_desc_scales(xs_base), ws_desc0 = umma_desc_scales(ws_base);
        bool ok = true;
        int i = 0, step = 0;
        for (int u = blockIdx.x; u < units; u += gridDim.x, ++i) {
            int m0, n0, k0, n;
            unit(u, m0, n0, k0, n);
            // the drain warps are done with this accumulator's previous tile
            if (i >= T::ACCS) ok = mbar_wait_polite(acc_empty0 + 8 * b.at, b.round ^ 1, wait_limit_ns, 0);
            const uint32_t acc = tmem + b.at * T::ACC_COLS;
            for (int k = 0; k < n; ++k, ++step) {
                ok = ok && mbar_wait_polite(full0 + 8 * s.at, s.round, wait_limit_ns, 0);
                // the place of this step's scales has been read by the products of the step before the last
                if (step >= 2) {
                    ok = ok && mbar_wait_polite(empty0 + 8 * before.at, before.round, wait_limit_ns, 0);
                    before.next();
                }
                if (!__all_sync(0xffffffffu, ok)) break;
                tc_fence_after_sync();
                if (elect_one()) {
                    const uint64_t w = w_desc0 + s.at * (T::W_BYTES >> 4), x = x_desc0 + s.at * (T::X_BYTES >> 4);
                    const uint64_t ws = ws_desc0 + s.at * (T::WS_BYTES >> 4), xs = xs_desc0 + s.at * (T::XS_BYTES >> 4);
                    const uint32_t w_scales = tmem + T::SCALES + (step & 1) * T::SCALE_COLS, x_scales = w_scales + 4 * T::KT;
                    // products of 64 columns; the last step may have fewer
                    const int products = min(T::BK / 64, (p.K - (k0 + k) * T::BK + 63) / 64);
#pragma unroll
                    for (int t = 0; t < T::KT; ++t) {
                        if (t * (BLOCK / 16) >= products) break;
                        tmem_copy_scales(w_scales + 4 * t, ws + t * (kFp4TileBytes >> 4));
#pragma unroll
                        for (int r = 0; r < T::XT; ++r)
                            tmem_copy_scales(x_scales + 4 * (T::XT * t + r), xs + (r * T::KT + t) * (kFp4TileBytes >> 4));
                    }
                    const uint32_t x_first = TOK % 128 ? (uint32_t)(m0 % 128 / 32) : 0u;
#pragma unroll
                    for (int kk = 0; kk < T::BK / 64; ++kk) {
                        if (kk >= products) break;
                        const int t = kk / (BLOCK / 16);
                        umma_fp4<BLOCK>(acc, w + 2 * kk, x + 2 * kk, BLOCK == 32 && kk % 2 ? T::IDESC | T::SECOND_PAIR : T::IDESC,
                                        w_scales + 4 * t, x_scales + 4 * T::XT * t + x_first, kk > 0 || k > 0);
                    }
                    umma_commit(empty0 + 8 * s.at);  // the stage may be refilled once these have read it
                    // the tile is final once its products are done
                    if (k + 1 == n) umma_commit(acc_full0 + 8 * b.at);
                }
                __syncwarp();
                s.next();
            }
            if (!__all_sync(0xffffffffu, ok)) {
                *abort_flag = 1;
                break;
            }
            b.next();
        }
        // every product issued above has completed before the block moves on
        if (elect_one()) umma_commit(drained);
        __syncwarp();
        (void)mbar_wait_polite(drained, 0, wait_limit_ns, 0);
    } else {
        // drain warps: a lane is a row of B (a column of C), a column of the accumulator a token
        griddep_wait();  // the tokens' scales
        const int q = warp & 3;
        RingPlace<T::ACCS> b;
        for (int u = blockIdx.x; u < units; u += gridDim.x, b.next()) {
            int m0, n0, k0, n;
            unit(u, m0, n0, k0, n);
            const int col = n0 + 32 * q + lane;
            const bool in = col < p.N;
            // the scales are here before the accumulator is: lane l holds those of tokens l, l + 32, ...
            float token_scales[(TOK + 31) / 32];
#pragma unroll
            for (int i = 0; i < (TOK + 31) / 32; ++i) {
                const int m = m0 + 32 * i + lane;
                token_scales[i] = p.a_scale && m < p.M ? p.a_scale[m] : 1.f;
            }
            const float scale = in && p.b_scale ? p.b_scale[col] : 1.f, bias = in && p.bias ? p.bias[col] : 0.f;
            // a finished tile is stored whatever another role decided since
            if (!mbar_wait_warp(acc_full0 + 8 * b.at, b.round, wait_limit_ns, 200)) {
                if (lane == 0) *abort_flag = 1;
                break;
            }
            tc_fence_after_sync();
            const uint32_t acc = tmem + ((uint32_t)(32 * q) << 16) + b.at * T::ACC_COLS;
            constexpr int CHUNK = TOK % 32 ? 16 : 32;
#pragma unroll 1
            for (int c0 = 0; c0 < TOK; c0 += CHUNK) {
                float v[32];
                if constexpr (CHUNK == 32) tmem_ld32(acc + (uint32_t)c0, v);
                else tmem_ld16(acc + (uint32_t)c0, v);
                if (c0 + CHUNK == TOK) {
                    // the accumulator is read: hand it back to the product thread
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(acc_empty0 + 8 * b.at);
                }
                const int m = m0 + c0, count = min(CHUNK, p.M - m);
                if (count <= 0) continue;
                if (splits > 1) {
                    // the ring's copies have landed and been read: its first bytes hold this block's part
                    float *part = reinterpret_cast<float *>(smem) + 32 * q + lane;
#pragma unroll
                    for (int j = 0; j < CHUNK; ++j) part[(c0 + j) * T::ROWS] = v[j];
                    continue;
                }
                float token_scale = token_scales[0];
#pragma unroll
                for (int i = 1; i < (TOK + 31) / 32; ++i)
                    if (c0 / 32 == i) token_scale = token_scales[i];
#pragma unroll
                for (int j = 0; j < CHUNK; ++j) {
                    const float s = __shfl_sync(0xffffffffu, token_scale, c0 % 32 + j);
                    v[j] = fmaf(v[j] * s, scale, bias);
                }
                if (in) {
                    const int64_t at = (int64_t)m * p.ldc + col;
                    if (p.ctype == SGEMM_F32) {
#pragma unroll
                        for (int j = 0; j < CHUNK; ++j)
                            if (j < count) static_cast<float *>(p.C)[at + j * p.ldc] = v[j];
                    } else if (p.ctype == SGEMM_BF16) {
#pragma unroll
                        for (int j = 0; j < CHUNK; ++j)
                            if (j < count) static_cast<__nv_bfloat16 *>(p.C)[at + j * p.ldc] = __float2bfloat16_rn(v[j]);
                    } else {
#pragma unroll
                        for (int j = 0; j < CHUNK; ++j)
                            if (j < count) static_cast<__half *>(p.C)[at + j * p.ldc] = __float2half_rn(v[j]);
                    }
                }
            }
        }
    }

    __syncwarp();
    if (splits > 1) {
        cluster_sync();
        if (warp >= T::DRAIN) {
            // this block's tokens of the tile: the parts in order of their rank
            int m0, n0, k0, n;
            unit(blockIdx.x, m0, n0, k0, n);
            const int row = 32 * (warp & 3) + lane, col = n0 + row;
            const float scale = col < p.N && p.b_scale ? p.b_scale[col] : 1.f, bias = col < p.N && p.bias ? p.bias[col] : 0.f;
            for (int j = blockIdx.x % splits; j < TOK && m0 + j < p.M; j += splits) {
                float sum = 0.f;
#pragma unroll 4
                for (int r = 0; r < splits; ++r)
                    sum += __uint_as_float(dsmem_ld_u32(dsmem_map(base + 4 * (j * T::ROWS + row), (uint32_t)r)));
                const float s = p.a_scale ? p.a_scale[m0 + j] : 1.f;
                if (col < p.N) store_c(p.C, (int64_t)(m0 + j) * p.ldc + col, p.ctype, fmaf(sum * s, scale, bias));
            }
        }
        cluster_sync();  // no block leaves while another reads its part
    }
    tc_fence_before_sync();
    __syncthreads();
    if (*abort_flag && tid == 0) {
        atomicCAS(err_word, 0, 1);
        // let the copies still in flight land before shared memory is released (bounded)
        for (int t = issued - T::STAGES > 0 ? issued - T::STAGES : 0; t < issued; ++t)
            (void)mbar_wait_polite(full0 + 8 * (t % T::STAGES), (t / T::STAGES) & 1, wait_limit_ns, 0);
    }
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 0) tmem_dealloc(tmem, T::TMEM_COLS);
}

// The product over no columns: the bias, or 0.
__global__ void __launch_bounds__(256) fp4_empty_kernel(const Fp4Args p) {
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < (int64_t)p.M * p.N; i += (int64_t)gridDim.x * blockDim.x)
        store_c(p.C, i / p.N * p.ldc + i % p.N, p.ctype, p.bias ? p.bias[i % p.N] : 0.f);
}

}  // namespace sgemm
