// The product of 4-bit operands for many tokens: pairs of SMs on one tile.
//
// Tiles of 128 rows of B by 192 or 256 tokens on one SM (fp4_mma.cuh) need more of L2
// than it gives: 8192 x 8192 x 8192 takes 250 - 280 us, and 210 with a quarter of the
// products left out.  A pair's tile has 256 rows of B, 128 in each SM, and its
// tcgen05.mma (cta_group::2) reads the tokens' codes from both SMs' shared memory, half
// of them each, so a product of the same size copies a third less.
//
// The blocks of a pair copy their own halves, announced to the first block's barriers;
// its product warp issues for both, and the commits reach the barriers of both.  Each
// block drains the accumulator of its own 128 rows: sixteen warps take 64 columns of 32 rows
// each into registers, so that the next tile's products, which need the same columns of
// tensor memory, wait for little more than that.
//
// 8192 x 8192 x 8192 takes 164 us with blocks of 16 and 151 with blocks of 32, 6.7 and 7.3
// PFLOP/s: 14 rounds of 76 tiles where 13.5 would do, of 32 steps of some 610 cycles (the
// products of one take 512 in instructions of 64 columns; PTX has one of 96 for this chip, at up
// to 1.5 times the rate, which is not used) and some 1000 to hand the accumulator over, at the 1.73 GHz that
// the power cap leaves.  Short K is bound by what a round stores: 4864 x 4096 x 512 with
// BF16 results 14.0 us, some 4500 cycles a round; FP32 results leave at 23 bytes a cycle and SM,
// as fast as a fill writes them.
#pragma once

#include <cuda.h>

#include <cstdint>
#include <type_traits>

#include "fp4_mma.cuh"
#include "ptx.cuh"
#include "tcgen05.cuh"
#include "tile_map.cuh"

namespace sgemm {

// ---------------------------------------------------------------- the forms for pairs of blocks

__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(dst), "r"(ncols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;\n" ::"r"(taddr), "r"(ncols) : "memory");
}

// tma_load_2d into this block's shared memory, completing on a barrier of either block of the pair.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const void *tensor_map, int x, int y, uint32_t cluster_bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];\n" ::"r"(dst),
        "l"(tensor_map), "r"(x), "r"(y), "r"(cluster_bar)
        : "memory");
}

// Arrive once on the barrier at this offset in both blocks when every product issued so far is done.
__device__ __forceinline__ void umma_commit_pair(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}

// One plain arrival on a barrier of a block of the cluster, which hands over tensor memory that was read
// and nothing that was written: with release semantics it would wait for the thread's stores, those of
// the tile before (1000 to 2000 cycles a tile; 8192 x 8192 x 8192 179 us, so 171).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n" ::"r"(cluster_bar) : "memory");
}

// umma_fp4 and tmem_copy_scales on a pair: A's rows and D's lanes are half in each block, B's rows too.
template <int BLOCK>
__device__ __forceinline__ void umma_fp4_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                              uint32_t a_scale, uint32_t b_scale, uint32_t accumulate) {
    if constexpr (BLOCK == 16)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(
                d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(a_scale), "r"(b_scale), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(
                d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(a_scale), "r"(b_scale), "r"(accumulate)
            : "memory");
}
__device__ __forceinline__ void tmem_copy_scales_pair(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n" ::"r"(taddr), "l"(desc) : "memory");
}

// ---------------------------------------------------------------- results

// fp4_store of 16-bit numbers whose rows start on 4 bytes, by whole warps: two lanes, which have
// two columns of two tokens, exchange one each, so that a lane stores both columns of a token.
// left: the columns from this lane pair's first to C's end.  4864 x 4096 x 512 BF16 15.4 us, so 13.8 (weights in L2);
// the four and eight warps that drain on single SMs lose by it what it saves (3001 x 5000 x 512 15.7 us, 17.1).
template <int COLS, class T>
__device__ __forceinline__ void fp4_store_pairs(T *c, int64_t ldc, const float *v, const float *token_scales, float scale, float bias,
                                                int count, int left) {
    const bool odd = threadIdx.x & 1;
    const uint32_t take = odd ? 0x3276u : 0x5410u;  // the upper halves, the neighbour's first; the lower, the own first
    // exchanged first, sixteen tokens' at a time, and then stored: one by one each would wait for the other
#pragma unroll
    for (int g = 0; g < COLS; g += 16) {
        uint32_t both[8];
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const float4 f = *reinterpret_cast<const float4 *>(token_scales + g + 2 * i);
            const float s[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int j = g + 2 * (i + h);
                const float x = fmaf(v[j] * s[2 * h], scale, bias), y = fmaf(v[j + 1] * s[2 * h + 1], scale, bias);
                if constexpr (std::is_same_v<T, __half>) {
                    const __half2 w = __floats2half2_rn(x, y);
                    both[i + h] = *reinterpret_cast<const uint32_t *>(&w);
                } else {
                    const __nv_bfloat162 w = __floats2bfloat162_rn(x, y);
                    both[i + h] = *reinterpret_cast<const uint32_t *>(&w);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) both[i] = __byte_perm(both[i], __shfl_xor_sync(0xffffffffu, both[i], 1), take);
        if (left > 1) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (g + 2 * i + odd < count) *reinterpret_cast<uint32_t *>(c + (int64_t)(2 * i) * ldc) = both[i];
        } else if (left > 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (g + 2 * i + odd < count) *reinterpret_cast<uint16_t *>(c + (int64_t)(2 * i) * ldc) = (uint16_t)both[i];
        }
        __syncwarp();
        c += 16 * ldc;
    }
}
template <int COLS>
__device__ __forceinline__ void fp4_store_warp(const Fp4Args &p, const float *v, const float *token_scales, float scale, float bias,
                                               int m, int col) {
    if (p.ctype != SGEMM_F32 && p.ldc % 2 == 0 && (reinterpret_cast<uintptr_t>(p.C) & 3) == 0) {
        const int odd = threadIdx.x & 1, count = p.M - m, left = p.N - (col - odd);
        const int64_t at = (int64_t)(m + odd) * p.ldc + (col - odd);
        if (p.ctype == SGEMM_BF16)
            fp4_store_pairs<COLS>(static_cast<__nv_bfloat16 *>(p.C) + at, p.ldc, v, token_scales, scale, bias, count, left);
        else fp4_store_pairs<COLS>(static_cast<__half *>(p.C) + at, p.ldc, v, token_scales, scale, bias, count, left);
    } else if (col < p.N) {
        fp4_store<COLS>(p, v, token_scales, scale, bias, m, col);
    }
}

// ---------------------------------------------------------------- the kernel

template <int BLOCK_>
struct Fp4PairTile {
    static constexpr int ROWS = 256, TOK = 256, BLOCK = BLOCK_;  // of the pair: two rows of tiles of scales, 64 columns a load
    static constexpr int BK = 256, BYTES = BK / 2;
    static constexpr int DRAIN = 4, DRAIN_WARPS = 16, COLS = TOK / 4, THREADS = 32 * (DRAIN + DRAIN_WARPS);
    static constexpr int KT = BK / BLOCK / 4;
    // a stage of one block: its rows of B, its half of the tokens, their scales (of all tokens)
    static constexpr int W_BYTES = ROWS / 2 * BYTES, X_BYTES = TOK / 2 * BYTES;
    static constexpr int WS_BYTES = KT * kFp4TileBytes, XS_BYTES = 2 * WS_BYTES;
    static constexpr int STAGE = W_BYTES + X_BYTES + WS_BYTES + XS_BYTES;
    // the ring, the tokens' scales of each drain warp, barriers
    static constexpr int SCALE_BYTES = 4 * DRAIN_WARPS * COLS;
    static constexpr int STAGES = (227 * 1024 - 1024 - 256 - SCALE_BYTES) / STAGE;
    static constexpr int SMEM_BYTES = STAGES * STAGE + SCALE_BYTES + 1024 + 256;
    // tensor memory: the accumulator, then a place for the scales of each stage
    static constexpr int SCALES = TOK, SCALE_COLS = 4 * KT * 3, TMEM_COLS = 512;
    static constexpr uint32_t IDESC = (1u << 7) | (1u << 10) | ((uint32_t)(TOK >> 3) << 17) |
                                      ((BLOCK == 32 ? 1u : 0u) << 23) | ((uint32_t)(ROWS >> 4) << 24);
    static constexpr uint32_t SECOND_PAIR = (2u << 4) | (2u << 29);
    static_assert(STAGES >= 4 && STAGES <= 8 && SCALES + STAGES * SCALE_COLS <= TMEM_COLS, "a ring, and tensor memory");
};

// Pair b (blocks 2 b and 2 b + 1, a cluster) takes tiles b, b + pairs, ...  tmWS, tmXS: the
// scales' tiles, a row of tiles a row, in elements of 8 bytes.
template <int BLOCK>
__global__ void __launch_bounds__(Fp4PairTile<BLOCK>::THREADS, 1)
    fp4_pair_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                    const __grid_constant__ CUtensorMap tmWS, const __grid_constant__ CUtensorMap tmXS, const Fp4Args p,
                    int *__restrict__ err_word, unsigned long long wait_limit_ns, int debug) {
    using T = Fp4PairTile<BLOCK>;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    unsigned char *smem = smem_raw + (base - raw);
    const uint32_t w_base = base + T::STAGES * T::X_BYTES, ws_base = w_base + T::STAGES * T::W_BYTES;
    const uint32_t xs_base = ws_base + T::STAGES * T::WS_BYTES;
    const uint32_t scales_base = xs_base + T::STAGES * T::XS_BYTES, bars = scales_base + T::SCALE_BYTES;
    // copies of both blocks done (of the first block), stage read by the products; accumulator final,
    // accumulator read by both (of the first block)
    const uint32_t full0 = bars, empty0 = full0 + 8 * T::STAGES;
    const uint32_t acc_full = empty0 + 8 * T::STAGES, acc_empty = acc_full + 8, drained = acc_empty + 8;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + (drained + 8 - base));
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + (drained + 12 - base));

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_ctarank();
    const int tiles_n = (p.N + T::ROWS - 1) / T::ROWS, tiles_m = (p.M + T::TOK - 1) / T::TOK, tiles = tiles_m * tiles_n;
    const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;
    const int steps = (p.K + T::BK - 1) / T::BK;
    auto tile = [&](int u, int &m0, int &n0) {
        int tn, tm;
        grouped_tile<8>(u, tiles_n, tiles_m, tn, tm);
        m0 = tm * T::TOK;
        n0 = tn * T::ROWS;
    };

    if (warp == 0) tmem_alloc_pair(smem_addr(tmem_slot), T::TMEM_COLS);
    if (tid == 32) {
        for (int s = 0; s < T::STAGES; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        mbar_init(acc_full, 1);
        mbar_init(acc_empty, 2 * T::DRAIN_WARPS);
        mbar_init(drained, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync();  // the other block's barriers exist
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;

    int issued = 0;  // copies: k-steps issued over all of this block's tiles
    if (warp == 0) {
        RingPlace<T::STAGES> s;
        const uint32_t first_full0 = dsmem_map(full0, 0);
        if (lane == 0) {
            prefetch_tensor_map(&tmW);
            prefetch_tensor_map(&tmX);
            prefetch_tensor_map(&tmWS);
            prefetch_tensor_map(&tmXS);
        }
        auto copy_b = [&](uint32_t at, int k, int n0) {
            if (elect_one()) {
                if (rank == 0) mbar_arrive_expect_tx(full0 + 8 * at, 2 * T::STAGE);
                tma_load_2d_pair(w_base + at * T::W_BYTES, &tmW, k * T::BYTES, n0 + (int)rank * (T::ROWS / 2), first_full0 + 8 * at);
                tma_load_2d_pair(ws_base + at * T::WS_BYTES, &tmWS, k * (T::WS_BYTES / 8), n0 / 128 + (int)rank, first_full0 + 8 * at);
            }
        };
        auto copy_tokens = [&](uint32_t at, int k, int m0) {
            if (elect_one()) {
                tma_load_2d_pair(base + at * T::X_BYTES, &tmX, k * T::BYTES, m0 + (int)rank * (T::TOK / 2), first_full0 + 8 * at);
                tma_load_2d_pair(xs_base + at * T::XS_BYTES, &tmXS, k * (T::WS_BYTES / 8), m0 / 128, first_full0 + 8 * at);
            }
        };
        // The tokens' codes may come from the kernel before; B does not: the first tile's first stages
        // of it are on their way before that kernel is waited for.
        int ahead = 0, m0, n0;
        if (!(debug & 1) && pair < tiles) {
            tile(pair, m0, n0);
            for (ahead = min(steps, T::STAGES); issued < ahead; ++issued) copy_b(issued, issued, n0);
        }
        griddep_wait();
        for (int k = 0; k < ahead; ++k, s.next()) copy_tokens(k, k, m0);
        bool ok = true;
        for (int u = pair; ok && !(debug & 1) && u < tiles; u += pairs) {
            tile(u, m0, n0);
            for (int k = u == pair ? ahead : 0; k < steps; ++k) {
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
    } else if (warp == 1 && rank == 0) {
        // One lane walks the steps: what it spends on one, beside the 512 cycles that the products take,
        // bounds the kernel.  (With the whole warp, a vote a step, two places for the scales and a wait
        // for each, a step took 760 cycles of issue alone.)
        if (elect_one()) {
            RingPlace<T::STAGES> s;
            const uint64_t x_desc0 = umma_desc_128b(base), w_desc0 = umma_desc_128b(w_base);
            const uint64_t xs_desc0 = umma_desc_scales(xs_base), ws_desc0 = umma_desc_scales(ws_base);
            // The scales' and codes' products of a step of N times 64 columns.  The scales have a place for each
            // stage: it was read by the time that the stage was refilled.
            auto issue = [&](bool first, auto n_const) {
                constexpr int N = decltype(n_const)::value;
                const uint64_t w = w_desc0 + s.at * (T::W_BYTES >> 4), x = x_desc0 + s.at * (T::X_BYTES >> 4);
                const uint64_t ws = ws_desc0 + s.at * (T::WS_BYTES >> 4), xs = xs_desc0 + s.at * (T::XS_BYTES >> 4);
                const uint32_t w_scales = tmem + T::SCALES + s.at * T::SCALE_COLS, x_scales = w_scales + 4 * T::KT;
#pragma unroll
                for (int t = 0; t * (BLOCK / 16) < N; ++t) {
                    tmem_copy_scales_pair(w_scales + 4 * t, ws + t * (kFp4TileBytes >> 4));
#pragma unroll
                    for (int r = 0; r < 2; ++r)
                        tmem_copy_scales_pair(x_scales + 4 * (2 * t + r), xs + (r * T::KT + t) * (kFp4TileBytes >> 4));
                }
#pragma unroll
                for (int kk = 0; kk < N; ++kk) {
                    const int t = kk / (BLOCK / 16);
                    umma_fp4_pair<BLOCK>(tmem, w + 2 * kk, x + 2 * kk, BLOCK == 32 && kk % 2 ? T::IDESC | T::SECOND_PAIR : T::IDESC,
                                         w_scales + 4 * t, x_scales + 8 * t, kk > 0 || !first);
                }
                umma_commit_pair(empty0 + 8 * s.at);
            };
            const int last = (p.K - (steps - 1) * T::BK + 63) / 64;  // products of the last step
            bool ok = true, ready = false;
            uint32_t turn = 0;  // of the accumulator: the parity of the tiles before
            for (int u = pair; ok && u < tiles; u += pairs, turn ^= 1) {
                if (u != pair) ok = mbar_wait_polite(acc_empty, turn ^ 1, wait_limit_ns, 0);
                for (int k = 0; ok && k < steps; ++k) {
                    if (!ready && !(ok = mbar_wait_polite(full0 + 8 * s.at, s.round, wait_limit_ns, 0))) break;
                    tc_fence_after_sync();
                    RingPlace<T::STAGES> next = s;
                    next.next();
                    ready = mbar_try_wait(full0 + 8 * next.at, next.round);  // asked early, looked at next time
                    if (k + 1 < steps || last == 4) issue(k == 0, std::integral_constant<int, 4>{});
                    else if (last == 3) issue(k == 0, std::integral_constant<int, 3>{});
                    else if (last == 2) issue(k == 0, std::integral_constant<int, 2>{});
                    else issue(k == 0, std::integral_constant<int, 1>{});
                    if (k + 1 == steps) umma_commit_pair(acc_full);
                    s = next;
                }
            }
            if (!ok) *abort_flag = 1;
            umma_commit_pair(drained);
        }
        __syncwarp();
        // every product issued above has completed before the pair moves on
        (void)mbar_wait_polite(drained, 0, wait_limit_ns, 0);
    } else if (warp == 1) {
        // commits reach this block too: it stays until the last one has
        (void)mbar_wait_warp(drained, 0, wait_limit_ns, 1000);
    } else if (warp >= T::DRAIN) {
        // drain warps: a lane is a row of B (a column of C), a column of the accumulator a token
        griddep_wait();  // the tokens' scales
        const int q = warp & 3, c0 = (warp - T::DRAIN) / 4 * T::COLS;
        float *token_scales = reinterpret_cast<float *>(smem + (scales_base - base)) + (warp - T::DRAIN) * T::COLS;
        uint32_t turn = 0;
        for (int u = pair; u < tiles; u += pairs, turn ^= 1) {
            int m0, n0;
            tile(u, m0, n0);
            m0 += c0;
            const int col = n0 + (int)rank * (T::ROWS / 2) + 32 * q + lane;
            const bool in = col < p.N;
            // the scales are here before the accumulator is
#pragma unroll
            for (int j = lane; j < T::COLS; j += 32) token_scales[j] = p.a_scale && m0 + j < p.M ? p.a_scale[m0 + j] : 1.f;
            const float scale = in && p.b_scale ? p.b_scale[col] : 1.f, bias = in && p.bias ? p.bias[col] : 0.f;
            if (!mbar_wait_warp(acc_full, turn, wait_limit_ns, 20)) {
                if (lane == 0) *abort_flag = 1;
                break;
            }
            tc_fence_after_sync();
            float v[T::COLS];
            tmem_ld64(tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)c0, v);
            // the accumulator is read: hand it back to the product warp
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(dsmem_map(acc_empty, 0));
            fp4_store_warp<T::COLS>(p, v, token_scales, scale, bias, m0, col);
            __syncwarp();  // the scales are read before the next tile's take their place
        }
    }

    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    if (*abort_flag && tid == 0) {
        atomicCAS(err_word, 0, 1);
        // let the copies still in flight land before shared memory is released (bounded); they are
        // counted by the first block's barriers
        if (rank == 0)
            for (int t = issued - T::STAGES > 0 ? issued - T::STAGES : 0; t < issued; ++t)
                (void)mbar_wait_polite(full0 + 8 * (t % T::STAGES), (t / T::STAGES) & 1, wait_limit_ns, 0);
    }
    __syncthreads();
    cluster_sync();  // neither block leaves while the other's products, commits or arrivals are on their way
    tc_fence_after_sync();
    if (warp == 0) tmem_dealloc_pair(tmem, T::TMEM_COLS);
}

}  // namespace sgemm
