// The product of 4-bit operands with block scales on the 5th-generation tensor
// cores: tcgen05.mma multiplies the codes, scales the products of each block and
// adds them up in FP32; the rows' scales and the bias follow when the accumulator
// is drained.
//
// A tile is 128 rows of B, the weights, by up to 128 tokens, transposed: lanes of
// tensor memory are rows of B, columns tokens.  A k-step is 256 columns, 128 bytes
// of codes a row, which TMA copies into swizzled rows; the scales, already laid out
// in tiles of 512 bytes (fp4_quantize.cuh), follow as plain bulk copies and go on
// into tensor memory by tcgen05.cp, issued in front of the products that use them.
//
// One block per SM walks tiles: one thread copies into a ring, one issues, four or
// eight warps drain.  Where there are few tiles, a cluster of blocks shares each: every
// block adds up a part of K and the parts are joined through distributed shared
// memory, in a fixed order.  Every wait is bounded; a block that gives up records an
// error code and frees its tensor memory.
//
// Few tokens wait for one block's chain of steps: one of up to 128 tokens lasts 395 to 450
// cycles, those of issuing twelve instructions and their way through the pipe, where the
// products alone need 64 to 256.  24 x 4096 x 4096 takes 7.8 us with weights in turn, from HBM
// (7.5 with the same ones in L2), 24 x 16384 x 4096, whose 36 MB need 5.3, 10.6 (7.7); 64 to
// 512 tokens by 4096 x 4096 take 8.4 to 9.2 whatever their number.
#pragma once

#include <cuda.h>

#include <cstdint>
#include <type_traits>

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

// Stores COLS columns of an accumulator: column j is token m + j of column `col` of C, whose row of B
// this lane is.  token_scales: those of the COLS tokens, in shared memory (read four at a time by
// the whole warp; exchanged between lanes they were a chain of latencies: 4096 x 4096 x 512, of which
// storing is the most, 31 us against 24).
template <int COLS, class T>
__device__ __forceinline__ void fp4_store_as(T *c, int64_t ldc, const float *v, const float *token_scales, float scale, float bias,
                                             int count) {
    constexpr int DT = sizeof(T) == 4 ? SGEMM_F32 : std::is_same_v<T, __half> ? SGEMM_F16 : SGEMM_BF16;
#pragma unroll
    for (int j = 0; j < COLS; j += 4) {
        const float4 f = *reinterpret_cast<const float4 *>(token_scales + j);
        const float s[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
        for (int i = 0; i < 4; ++i, c += ldc)
            if (j + i < count) *c = Elem<DT>::from_float(fmaf(v[j + i] * s[i], scale, bias));
    }
}
template <int COLS>
__device__ __forceinline__ void fp4_store(const Fp4Args &p, const float *v, const float *token_scales, float scale, float bias,
                                          int m, int col) {
    const int64_t at = (int64_t)m * p.ldc + col;
    const int count = p.M - m;
    if (p.ctype == SGEMM_F32) fp4_store_as<COLS>(static_cast<float *>(p.C) + at, p.ldc, v, token_scales, scale, bias, count);
    else if (p.ctype == SGEMM_BF16)
        fp4_store_as<COLS>(static_cast<__nv_bfloat16 *>(p.C) + at, p.ldc, v, token_scales, scale, bias, count);
    else fp4_store_as<COLS>(static_cast<__half *>(p.C) + at, p.ldc, v, token_scales, scale, bias, count);
}

template <int TOK_, int BLOCK_>
struct Fp4Tile {
    static constexpr int ROWS = 128, TOK = TOK_, BLOCK = BLOCK_;
    static constexpr int BK = 256, BYTES = BK / 2;  // a k-step's columns, and bytes of codes a row
    // warps: 0 copies, 1 products, then sets of four that drain; a set takes COLS tokens of a tile
    static constexpr int SETS = TOK > 64 ? 2 : 1, COLS = TOK / SETS, DRAIN = 2, THREADS = 32 * (DRAIN + 4 * SETS);
    // 512-byte tiles of scales along a k-step; the tokens are in one row of tiles, from a multiple of 64
    // on: a product's scales start on an even column of tensor memory.  Narrower tiles serve only where
    // one holds all tokens.
    static constexpr int KT = BK / BLOCK / 4;
    static constexpr int W_BYTES = ROWS * BYTES, X_BYTES = TOK * BYTES;
    static constexpr int WS_BYTES = KT * kFp4TileBytes, XS_BYTES = WS_BYTES;
    static constexpr int STAGE = W_BYTES + X_BYTES + WS_BYTES + XS_BYTES;
    // tensor memory: accumulators, then a place for the scales of each stage
    static constexpr int ACCS = 2, ACC_COLS = TOK < 32 ? 32 : TOK;
    static constexpr int SCALES = ACCS * ACC_COLS, SCALE_COLS = 8 * KT, TMEM_COLS = 512;
    static constexpr int FIT_SMEM = (227 * 1024 - 1024 - 256 - 16 * TOK) / STAGE, FIT_TMEM = (TMEM_COLS - SCALES) / SCALE_COLS;
    static constexpr int FIT = FIT_SMEM < FIT_TMEM ? FIT_SMEM : FIT_TMEM, STAGES = FIT < 8 ? FIT : 8;
    // the ring, the tokens' scales of each drain warp, barriers
    static constexpr int SMEM_BYTES = STAGES * STAGE + 16 * TOK + 1024 + 256;
    // A = B = e2m1 (1 at bits 7 and 10), both K-major, N >> 3 at bit 17, e8m0 scales at bit 23, M >> 4 at
    // bit 24; which pair of bytes of a scale's word is used, at bits 4 (B) and 29 (A)
    static constexpr uint32_t IDESC = (1u << 7) | (1u << 10) | ((uint32_t)(TOK >> 3) << 17) |
                                      ((BLOCK == 32 ? 1u : 0u) << 23) | ((uint32_t)(ROWS >> 4) << 24);
    static constexpr uint32_t SECOND_PAIR = (2u << 4) | (2u << 29);
    static_assert(TOK == 16 || TOK == 32 || TOK == 64 || TOK == 128, "columns of one product");
    static_assert(STAGES >= 4, "a ring that hides the copies");
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
    const uint32_t xs_base = ws_base + T::STAGES * T::WS_BYTES;
    const uint32_t scales_base = xs_base + T::STAGES * T::XS_BYTES, bars = scales_base + 16 * TOK;
    // copies done, stage read by the products; accumulator final, accumulator read
    const uint32_t full0 = bars, empty0 = full0 + 8 * T::STAGES;
    const uint32_t acc_full0 = empty0 + 8 * T::STAGES, acc_empty0 = acc_full0 + 8 * T::ACCS;
    const uint32_t drained = acc_empty0 + 8 * T::ACCS;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + (drained + 8 - base));
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + (drained + 12 - base));

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int tiles_n = (p.N + T::ROWS - 1) / T::ROWS, tiles_m = (p.M + TOK - 1) / TOK;
    const int units = tiles_m * tiles_n * splits;
    const int steps = (p.K + T::BK - 1) / T::BK, k_tiles = fp4_tiles(p.K, BLOCK);
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
            mbar_init(acc_empty0 + 8 * b, 4 * T::SETS);  // one arrival per drain warp
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
        auto copy_b = [&](uint32_t at, int k, int n0) {
            if (elect_one()) {
                const uint32_t kt = (uint32_t)min(T::KT, k_tiles - k * T::KT) * kFp4TileBytes;
                mbar_arrive_expect_tx(full0 + 8 * at, T::W_BYTES + T::X_BYTES + 2 * kt);
                tma_load_2d(w_base + at * T::W_BYTES, &tmW, k * T::BYTES, n0, full0 + 8 * at);
                bulk_load(ws_base + at * T::WS_BYTES, p.b_tiles + ((int64_t)(n0 / 128) * k_tiles + k * T::KT) * kFp4TileBytes,
                          kt, full0 + 8 * at);
            }
        };
        auto copy_tokens = [&](uint32_t at, int k, int m0) {
            if (elect_one()) {
                const uint32_t kt = (uint32_t)min(T::KT, k_tiles - k * T::KT) * kFp4TileBytes;
                tma_load_2d(base + at * T::X_BYTES, &tmX, k * T::BYTES, m0, full0 + 8 * at);
                bulk_load(xs_base + at * T::XS_BYTES, p.a_tiles + ((int64_t)(m0 / 128) * k_tiles + k * T::KT) * kFp4TileBytes,
                          kt, full0 + 8 * at);
            }
        };
        // The tokens' codes may come from the kernel before; B does not: the first unit's first stages
        // of it are on their way before that kernel is waited for.
        int ahead = 0, m0, n0, k0, n;
        if (!(debug & 1) && (int)blockIdx.x < units) {
            unit(blockIdx.x, m0, n0, k0, n);
            for (ahead = min(n, T::STAGES); issued < ahead; ++issued) copy_b(issued, k0 + issued, n0);
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
                copy_b(s.at, k, n0);
                copy_tokens(s.at, k, m0);
                __syncwarp();
                ++issued;
                s.next();
            }
        }
    } else if (warp == 1) {
        // one lane walks the steps: what it spends on one bounds the products of few tokens
        if (elect_one()) {
            RingPlace<T::STAGES> s;
            RingPlace<T::ACCS> b;
            const uint64_t x_desc0 = umma_desc_128b(base), w_desc0 = umma_desc_128b(w_base);
            const uint64_t xs_desc0 = umma_desc_scales(xs_base), ws_desc0 = umma_desc_scales(ws_base);
            // The scales' and codes' products of a step of N times 64 columns.  The scales have a place for each
            // stage: it was read by the time that the stage was refilled.
            auto issue = [&](uint32_t acc, uint32_t x_first, bool first, auto n_const) {
                constexpr int N = decltype(n_const)::value;
                const uint64_t w = w_desc0 + s.at * (T::W_BYTES >> 4), x = x_desc0 + s.at * (T::X_BYTES >> 4);
                const uint64_t ws = ws_desc0 + s.at * (T::WS_BYTES >> 4), xs = xs_desc0 + s.at * (T::XS_BYTES >> 4);
                const uint32_t w_scales = tmem + T::SCALES + s.at * T::SCALE_COLS, x_scales = w_scales + 4 * T::KT;
#pragma unroll
                for (int t = 0; t * (BLOCK / 16) < N; ++t) {
                    tmem_copy_scales(w_scales + 4 * t, ws + t * (kFp4TileBytes >> 4));
                    tmem_copy_scales(x_scales + 4 * t, xs + t * (kFp4TileBytes >> 4));
                }
#pragma unroll
                for (int kk = 0; kk < N; ++kk) {
                    const int t = kk / (BLOCK / 16);
                    umma_fp4<BLOCK>(acc, w + 2 * kk, x + 2 * kk, BLOCK == 32 && kk % 2 ? T::IDESC | T::SECOND_PAIR : T::IDESC,
                                    w_scales + 4 * t, x_scales + 4 * t + x_first, kk > 0 || !first);
                }
                umma_commit(empty0 + 8 * s.at);  // the stage may be refilled once these have read it
            };
            const int last = (p.K - (steps - 1) * T::BK + 63) / 64;  // products of the last step of K
            bool ok = true, ready = false;
            int i = 0;
            for (int u = blockIdx.x; ok && u < units; u += gridDim.x, ++i, b.next()) {
                int m0, n0, k0, n;
                unit(u, m0, n0, k0, n);
                // the drain warps are done with this accumulator's previous tile
                if (i >= T::ACCS) ok = mbar_wait_polite(acc_empty0 + 8 * b.at, b.round ^ 1, wait_limit_ns, 0);
                const uint32_t acc = tmem + b.at * T::ACC_COLS, x_first = TOK % 128 ? (uint32_t)(m0 % 128 / 32) : 0u;
                for (int k = 0; ok && k < n; ++k) {
                    if (!ready && !(ok = mbar_wait_polite(full0 + 8 * s.at, s.round, wait_limit_ns, 0))) break;
                    tc_fence_after_sync();
                    RingPlace<T::STAGES> next = s;
                    next.next();
                    ready = mbar_try_wait(full0 + 8 * next.at, next.round);  // asked early, looked at next time
                    if (k0 + k + 1 < steps || last == 4) issue(acc, x_first, k == 0, std::integral_constant<int, 4>{});
                    else if (last == 3) issue(acc, x_first, k == 0, std::integral_constant<int, 3>{});
                    else if (last == 2) issue(acc, x_first, k == 0, std::integral_constant<int, 2>{});
                    else issue(acc, x_first, k == 0, std::integral_constant<int, 1>{});
                    if (k + 1 == n) umma_commit(acc_full0 + 8 * b.at);  // the tile is final once its products are done
                    s = next;
                }
            }
            if (!ok) *abort_flag = 1;
            umma_commit(drained);
        }
        __syncwarp();
        // every product issued above has completed before the block moves on
        (void)mbar_wait_polite(drained, 0, wait_limit_ns, 0);
    } else {
        // drain warps: a lane is a row of B (a column of C), a column of the accumulator a token
        griddep_wait();  // the tokens' scales
        constexpr int COLS = T::COLS, LOAD = COLS < 32 ? 16 : COLS < 64 ? 32 : 64;
        const int q = warp & 3, c0 = (warp - T::DRAIN) / 4 * COLS;
        float *token_scales = reinterpret_cast<float *>(smem + (scales_base - base)) + (warp - T::DRAIN) * COLS;
        RingPlace<T::ACCS> b;
        for (int u = blockIdx.x; u < units; u += gridDim.x, b.next()) {
            int m0, n0, k0, n;
            unit(u, m0, n0, k0, n);
            m0 += c0;
            const int col = n0 + 32 * q + lane;
            const bool in = col < p.N;
            // the scales are here before the accumulator is
            for (int j = lane; j < COLS; j += 32) token_scales[j] = p.a_scale && m0 + j < p.M ? p.a_scale[m0 + j] : 1.f;
            const float scale = in && p.b_scale ? p.b_scale[col] : 1.f, bias = in && p.bias ? p.bias[col] : 0.f;
            // a finished tile is stored whatever another role decided since
            if (!mbar_wait_warp(acc_full0 + 8 * b.at, b.round, wait_limit_ns, 20)) {
                if (lane == 0) *abort_flag = 1;
                break;
            }
            tc_fence_after_sync();
            const uint32_t acc = tmem + ((uint32_t)(32 * q) << 16) + b.at * T::ACC_COLS + (uint32_t)c0;
            float v[LOAD];
            if constexpr (LOAD == 16) tmem_ld16(acc, v);
            else if constexpr (LOAD == 32) tmem_ld32(acc, v);
            else tmem_ld64(acc, v);
            // the accumulator is read: hand it back to the product thread
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(acc_empty0 + 8 * b.at);
            if (splits > 1) {
                // the ring's copies have landed and been read: its first bytes hold this block's part
                float *part = reinterpret_cast<float *>(smem) + c0 * T::ROWS + 32 * q + lane;
#pragma unroll
                for (int j = 0; j < COLS; ++j) part[j * T::ROWS] = v[j];
            } else if (in) {
                fp4_store<COLS>(p, v, token_scales, scale, bias, m0, col);
            }
            __syncwarp();  // the scales are read before the next tile's take their place
        }
    }

    __syncwarp();
    if (splits > 1) {
        cluster_sync();
        if (warp >= T::DRAIN) {
            // this block's tokens of the tile, a warp each and a lane four of its rows: the parts in order of
            // their rank, four tokens' on their way
            constexpr int U = 4, WARPS = 4 * T::SETS;
            int m0, n0, k0, n;
            unit(blockIdx.x, m0, n0, k0, n);
            const int tokens = min(TOK, p.M - m0), col = n0 + 4 * lane, step = splits * WARPS;
            float scale[4], bias[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                scale[i] = col + i < p.N && p.b_scale ? p.b_scale[col + i] : 1.f;
                bias[i] = col + i < p.N && p.bias ? p.bias[col + i] : 0.f;
            }
            for (int j = blockIdx.x % splits + (warp - T::DRAIN) * splits; j < tokens; j += U * step) {
                float4 sum[U] = {};
#pragma unroll 4
                for (int r = 0; r < splits; ++r) {
                    const uint32_t from = dsmem_map(base + 4 * (j * T::ROWS + 4 * lane), (uint32_t)r);
#pragma unroll
                    for (int i = 0; i < U; ++i) {
                        if (j + i * step >= tokens) break;
                        const ulonglong2 v = dsmem_ld_v2u64(from + 4 * T::ROWS * i * step);
                        const float2 lo = f32x2_unpack(v.x), hi = f32x2_unpack(v.y);
                        sum[i].x += lo.x, sum[i].y += lo.y, sum[i].z += hi.x, sum[i].w += hi.y;
                    }
                }
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    if (j + i * step >= tokens) break;
                    const int64_t m = m0 + j + i * step;
                    const float s = p.a_scale ? p.a_scale[m] : 1.f, v[4] = {sum[i].x, sum[i].y, sum[i].z, sum[i].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (col + e < p.N) store_c(p.C, m * p.ldc + col + e, p.ctype, fmaf(v[e] * s, scale[e], bias[e]));
                }
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
