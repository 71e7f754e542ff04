// The product of 8-bit operands on the 5th-generation tensor cores.  B, the
// weights, stays 8-bit on its way from memory: a tile of 128 rows of B is the
// A operand of tcgen05.mma, which converter warps write into tensor memory as
// FP16 (i8_codes.cuh), so that no FP16 copy of it ever reaches shared or global
// memory; up to 256 tokens' codes, FP16 in memory, are the B operand.  The FP32
// accumulators hold the transposed tile: lanes are rows of B, columns tokens.
//
// For few tokens the time is that of reading B once; for many it is the tensor
// cores' (2 M N K at the FP16 rate).  Per 64-deep k-step of a 128 x TOK tile
// shared memory sees 8 KB of B written and read once and TOK x 128 bytes of
// tokens written and read once: below the 128 bytes a cycle it can move, where
// B as FP16 in shared memory would be beyond it.
//
// Measured, with the kernel that quantises the tokens and, where K is split, the
// one that adds the splits: 24 x 16384 x 4096 18.5 - 19.4 us (3.6 TB/s of operands; two
// launches, one round of 128 tiles on 152 SMs, and the copies, the conversion
// and the products of a tile's first and last steps one after another);
// 4096 x 4096 x 4096 103 us; 8192 x 8192 x 8192 713 us, 1541 TFLOP/s, 79 % of what
// FP16 products reach: 48 us quantise, then the tensor pipe is 72 % busy, held
// up by the issue of a step's products (680 cycles a step, 512 of them the
// pipe's; two steps to a round of that loop took 731 us) and by drains that 256
// columns leave no second accumulator to hide.  3001 x 4999 x 2047 in FP32
// takes 76.2 us: about 12 for quantising rows of single floats, 4 rounds of
// tiles, and 60 MB of results that all SMs store at the same time.
//
// One block per SM walks units (tile, k-split): one thread copies by TMA into a
// ring, eight warps convert, one thread issues the products, four warps drain
// the accumulator, apply the scales and the bias and store.  Every wait is
// bounded; a block that gives up records an error code, stores nothing more and
// frees its tensor memory.
#pragma once

#include <cuda.h>

#include <cstdint>

#include "i8_codes.cuh"
#include "ptx.cuh"
#include "tcgen05.cuh"
#include "tile_map.cuh"

namespace sgemm {

template <int TOK_>
struct I8StreamTile {
    static constexpr int ROWS = 128, TOK = TOK_;
    // k-steps of 128 where a stage of them leaves room for four: fewer barriers a byte of B
    static constexpr int BK = TOK <= 128 ? 128 : 64;
    // warps: 0 copies, 1 products, then SETS sets of four that convert every SETS-th k-step, and
    // four that drain
    static constexpr int SETS = 2, CONVERT = 4, DRAIN = CONVERT + 4 * SETS, THREADS = 32 * (DRAIN + 4);
    static constexpr int W_BYTES = ROWS * BK, X_BOX = TOK * 128, X_BYTES = X_BOX * (BK / 64), STAGE = W_BYTES + X_BYTES;
    // a stage is shared memory for both operands and BK / 2 columns of tensor memory for the codes of B
    static constexpr int A_COLS = BK / 2;
    // accumulators: two where tensor memory has room for both beside four stages
    static constexpr int ACCS = TOK <= 192 ? 2 : 1;
    static constexpr int ACC_COLS = TOK < 32 ? 32 : TOK;
    static constexpr int FIT_SMEM = (227 * 1024 - 1024 - 256) / STAGE, FIT_TMEM = (512 - ACCS * ACC_COLS) / A_COLS;
    static constexpr int STAGES = FIT_SMEM < FIT_TMEM ? FIT_SMEM : FIT_TMEM;
    static constexpr int SMEM_BYTES = STAGES * STAGE + 1024 + 256;
    static constexpr int TMEM_COLS = 512;
    // D = FP32 (bits 4-5 = 1), A = B = FP16 (0), both K-major, N >> 3 at bit 17, M >> 4 at bit 24
    static constexpr uint32_t IDESC = (1u << 4) | ((uint32_t)(TOK >> 3) << 17) | ((uint32_t)(ROWS >> 4) << 24);
    static_assert(TOK % 16 == 0 && TOK >= 16 && TOK <= 256, "columns of one product");
    static_assert(STAGES >= 4 && STAGES >= SETS, "a ring that hides the copies, and no set two rounds ahead of another");
};

// A place in a ring of N, and the parity of the rounds made.
template <int N>
struct RingPlace {
    uint32_t at = 0, round = 0;
    __device__ void next() {
        if (++at == N) {
            at = 0;
            round ^= 1;
        }
    }
};

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(p));
    return p != 0;
}

// D[tmem] (+)= A[tmem] * B[smem desc]^T with FP16 inputs and FP32 accumulation.
__device__ __forceinline__ void umma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Descriptor of a K-major operand in 128-byte swizzled rows (8 rows = 1024 bytes).
__device__ __forceinline__ uint64_t umma_desc_128b(uint32_t saddr) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)1u << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1u << 46) | ((uint64_t)2u << 61);
}

// 32 columns of this thread's lane of tensor memory.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};\n" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

// Unit u is tile u % tiles, k-split u / tiles; tiles run over the tokens first
// within groups of eight tiles of rows, so that blocks at work together share
// both operands in L2.  With splits > 1 each unit writes its raw sums to its
// own M x ldp slab of `partials` and i8_join_kernel adds the slabs in order and
// applies the scales.  laid_out: the kernel before writes B too, not the tokens'
// codes alone.  debug: the test-only switches (bit 0: no copies, so that the
// waits run out).
template <int TOK>
__global__ void __launch_bounds__(I8StreamTile<TOK>::THREADS, 1)
    i8_stream_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const I8Args p,
                     int splits, float *__restrict__ partials, int64_t ldp, int laid_out, int *__restrict__ err_word,
                     unsigned long long wait_limit_ns, int debug) {
    using T = I8StreamTile<TOK>;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    unsigned char *smem = smem_raw + (base - raw);
    // tokens' stages first, then B's (128-byte swizzled boxes start on 1024 bytes), then the barriers
    const uint32_t w_base = base + T::STAGES * T::X_BYTES, bars = w_base + T::STAGES * T::W_BYTES;
    // copies done, codes converted, stage read by the products; accumulator final, accumulator read
    const uint32_t full0 = bars, a_full0 = full0 + 8 * T::STAGES, empty0 = a_full0 + 8 * T::STAGES;
    const uint32_t acc_full0 = empty0 + 8 * T::STAGES, acc_empty0 = acc_full0 + 8 * T::ACCS;
    const uint32_t drained = acc_empty0 + 8 * T::ACCS;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + (drained + 8 - base));
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + (drained + 12 - base));

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int tiles_n = (p.N + T::ROWS - 1) / T::ROWS, tiles_m = (p.M + TOK - 1) / TOK;
    const int tiles = tiles_m * tiles_n, units = tiles * splits;
    const int steps = (p.K + T::BK - 1) / T::BK;
    auto unit = [&](int u, int &m0, int &n0, int &k0, int &n) {
        int tn, tm;
        grouped_tile<8>(u % tiles, tiles_n, tiles_m, tn, tm);
        m0 = tm * TOK;
        n0 = tn * T::ROWS;
        const int s = u / tiles;
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
            mbar_init(a_full0 + 8 * s, 4);  // one arrival per converter warp of a set
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
    const uint32_t tmem = *tmem_slot, tmem_a = tmem + T::ACCS * T::ACC_COLS;

    int issued = 0;  // copies: k-steps issued over all of this block's units
    if (warp == 0) {
        RingPlace<T::STAGES> s;
        if (lane == 0) {
            prefetch_tensor_map(&tmW);
            prefetch_tensor_map(&tmX);
        }
        // Copies of step k of a unit into the ring's next stage: B's part, which announces both, and
        // the tokens'.
        auto copy_b = [&](uint32_t at, int k, int n0) {
            if (elect_one()) {
                mbar_arrive_expect_tx(full0 + 8 * at, T::STAGE);
                tma_load_2d(w_base + at * T::W_BYTES, &tmW, k * T::BK, n0, full0 + 8 * at);
            }
        };
        auto copy_tokens = [&](uint32_t at, int k, int m0) {
            if (elect_one())
#pragma unroll
                for (int h = 0; h < T::BK / 64; ++h)
                    tma_load_2d(base + at * T::X_BYTES + h * T::X_BOX, &tmX, k * T::BK + 64 * h, m0, full0 + 8 * at);
        };
        // The tokens' codes come from the kernel before, and B too where its rows had to be laid out.
        // The caller's own B does not: the first unit's first stages of it are on their way before
        // that kernel is waited for.
        int ahead = 0, m0, n0, k0, n;
        if (!laid_out && !(debug & 1) && (int)blockIdx.x < units) {
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
        // the whole warp walks the steps, so that addresses stay uniform; one lane issues
        RingPlace<T::STAGES> s;
        RingPlace<T::ACCS> b;
        const uint64_t x_desc0 = umma_desc_128b(base);
        bool ok = true;
        int i = 0;
        for (int u = blockIdx.x; u < units; u += gridDim.x, ++i) {
            int m0, n0, k0, n;
            unit(u, m0, n0, k0, n);
            // the drain warps are done with this accumulator's previous tile
            if (i >= T::ACCS) ok = mbar_wait_polite(acc_empty0 + 8 * b.at, b.round ^ 1, wait_limit_ns, 0);
            const uint32_t acc = tmem + b.at * T::ACC_COLS;
            for (int k = 0; k < n; ++k) {
                // the converters have seen the copies of both operands land
                ok = ok && mbar_wait_polite(a_full0 + 8 * s.at, s.round, wait_limit_ns, 0);
                if (!__all_sync(0xffffffffu, ok)) break;
                tc_fence_after_sync();
                if (elect_one()) {
                    const uint32_t w = tmem_a + s.at * T::A_COLS;
                    const uint64_t x = x_desc0 + s.at * (T::X_BYTES >> 4);
                    umma_f16_ta(acc, w, x, T::IDESC, k != 0);
#pragma unroll
                    for (int kk = 1; kk < T::BK / 16; ++kk)
                        umma_f16_ta(acc, w + kk * 8, x + (kk / 4) * (T::X_BOX >> 4) + (kk % 4) * 2, T::IDESC, 1);
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
    } else if (warp >= T::CONVERT && warp < T::DRAIN) {
        // converters: a warp takes the 32 rows of its quarter of tensor memory, in every SETS-th step,
        // so that a step's wait, reads and writes overlap the next ones'; the 16-byte pieces of a
        // lane's row are swizzled over 128 or 64 bytes
        const int row = 32 * (warp & 3) + lane, set = (warp - T::CONVERT) >> 2;
        const uint32_t to = tmem_a + ((uint32_t)(32 * (warp & 3)) << 16);
        const int swizzle = T::BK == 128 ? row & 7 : (row >> 1) & 3;
        RingPlace<T::STAGES> s;
        int turn = 0, step = 0;
        bool ok = true;
        for (int u = blockIdx.x; ok && u < units; u += gridDim.x) {
            int m0, n0, k0, n;
            unit(u, m0, n0, k0, n);
            for (int k = 0; k < n; ++k, ++step, s.next(), turn = turn + 1 == T::SETS ? 0 : turn + 1) {
                if (turn != set) continue;
                // A set sees only its own steps, and copies land in any order: it could reach a stage
                // whose previous copy is still on its way, where a wait for the phase after that one
                // would not wait at all.  So it first waits for the stage's previous products.  They
                // cannot be two rounds behind: the set's last step was SETS steps ago, all products
                // STAGES steps before that are done, and 2 STAGES >= SETS + STAGES.
                if (step >= T::STAGES) ok = mbar_wait_polite(empty0 + 8 * s.at, s.round ^ 1, wait_limit_ns, 20);
                ok = ok && mbar_wait_polite(full0 + 8 * s.at, s.round, wait_limit_ns, 20);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    *abort_flag = 1;
                    break;
                }
                const unsigned char *codes = smem + (w_base - base) + s.at * T::W_BYTES + row * T::BK;
#pragma unroll
                for (int h = 0; h < T::BK / 64; ++h) {
                    uint32_t r[32];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(codes + ((4 * h + c) ^ swizzle) * 16);
                        const uint2 q0 = i8x4_to_f16(v.x), q1 = i8x4_to_f16(v.y), q2 = i8x4_to_f16(v.z), q3 = i8x4_to_f16(v.w);
                        r[8 * c] = q0.x, r[8 * c + 1] = q0.y, r[8 * c + 2] = q1.x, r[8 * c + 3] = q1.y;
                        r[8 * c + 4] = q2.x, r[8 * c + 5] = q2.y, r[8 * c + 6] = q3.x, r[8 * c + 7] = q3.y;
                    }
                    if (h == 0) tc_fence_after_sync();
                    tmem_st32(to + s.at * T::A_COLS + 32 * h, r);
                }
                tmem_wait_st();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(a_full0 + 8 * s.at);
            }
        }
    } else if (warp >= T::DRAIN) {
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
            float scale = 1.f, bias = 0.f, token_scales[(TOK + 31) / 32];
#pragma unroll
            for (int i = 0; i < (TOK + 31) / 32; ++i) {
                const int m = m0 + 32 * i + lane;
                token_scales[i] = splits == 1 && m < p.M ? p.a_scale[m] : 0.f;
            }
            if (in && splits == 1) {
                scale = p.b_scale[col];
                if (p.bias) bias = p.bias[col];
            }
            // a finished tile is stored whatever another role decided since
            if (!mbar_wait_warp(acc_full0 + 8 * b.at, b.round, wait_limit_ns, 200)) {
                if (lane == 0) *abort_flag = 1;
                break;
            }
            tc_fence_after_sync();
            float *slab = splits > 1 ? partials + (int64_t)(u / tiles) * p.M * ldp : nullptr;
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
                if (slab) {
                    if (in)
#pragma unroll
                        for (int j = 0; j < CHUNK; ++j)
                            if (j < count) slab[(int64_t)(m + j) * ldp + col] = v[j];
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
    tc_fence_before_sync();
    __syncthreads();
    if (*abort_flag && tid == 0) {
        atomicCAS(err_word, 0, 1);
        // let the copies still in flight land before shared memory is released (bounded)
        for (int t = issued - T::STAGES > 0 ? issued - T::STAGES : 0; t < issued; ++t)
            (void)mbar_wait_polite(full0 + 8 * (t % T::STAGES), (t / T::STAGES) & 1, wait_limit_ns, 0);
    }
    if (*abort_flag && splits > 1 && warp >= T::DRAIN) {
        // this block's slabs are filled with NaN, so that no stale sums reach C
        for (int u = blockIdx.x; u < units; u += gridDim.x) {
            int m0, n0, k0, n;
            unit(u, m0, n0, k0, n);
            const int col = n0 + 32 * (warp & 3) + lane;
            if (col >= p.N) continue;
            for (int m = m0; m < min(m0 + TOK, p.M); ++m)
                partials[((int64_t)(u / tiles) * p.M + m) * ldp + col] = __int_as_float(0x7fc00000);
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 0) tmem_dealloc(tmem, T::TMEM_COLS);
}

// Adds the k-splits' slabs in order and applies the scales and the bias (with
// no split at all, K = 0, the sums are empty and the scales, which may not be
// finite or not exist, are not read).  blockIdx.y (+ gridDim.y, ...):
// rows of C; a thread four columns, whose sums lie on 16 bytes (ldp is a
// multiple of 4 and the slabs' rows are padded to it).
constexpr int kJoinThreads = 128;
__global__ void __launch_bounds__(kJoinThreads)
    i8_join_kernel(const I8Args p, int splits, const float *__restrict__ partials, int64_t ldp) {
    const int n = (blockIdx.x * kJoinThreads + threadIdx.x) * 4;
    if (n >= p.N) return;
    for (int64_t m = blockIdx.y; m < p.M; m += gridDim.y) {
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int k = 0; k < splits; ++k) {
            const float4 v = *reinterpret_cast<const float4 *>(partials + ((int64_t)k * p.M + m) * ldp + n);
            s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
        }
        const float sums[4] = {s.x, s.y, s.z, s.w}, scale = splits ? p.a_scale[m] : 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (n + i >= p.N) break;
            const float bias = p.bias ? p.bias[n + i] : 0.f;
            store_c(p.C, m * p.ldc + n + i, p.ctype, splits ? fmaf(sums[i] * scale, p.b_scale[n + i], bias) : bias);
        }
    }
}

}  // namespace sgemm
