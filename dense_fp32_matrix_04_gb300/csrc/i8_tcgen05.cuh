// The product of 8-bit operands on the 5th-generation tensor cores, for many
// rows of A: both operands as FP16 values (i8_codes.cuh), FP32 accumulators in
// tensor memory, the two scales and the bias applied as the tile is drained.
//
// Bound by the tensor cores: 2 M N K operations at the FP16 rate.  A persistent
// kernel of one block per SM walks 128 x BN tiles: one thread copies 64-deep
// k-steps of both operands by TMA into a ring of 128-byte swizzled rows, one
// thread issues the tcgen05.mma of 128 x BN x 16, and four warps drain the
// other of two accumulators meanwhile, so that copies, products and stores of
// neighbouring tiles overlap.  Every wait is bounded; a block that gives up
// records an error code, stores nothing more and frees its tensor memory.
#pragma once

#include <cuda.h>

#include <cstdint>

#include "i8_codes.cuh"
#include "ptx.cuh"
#include "tcgen05.cuh"
#include "tile_map.cuh"

namespace sgemm {

template <int BN_>
struct I8Tile {
    static constexpr int BM = 128, BN = BN_, BK = 64;
    static constexpr int THREADS = 192;  // copies, products, four drain warps
    static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128, STAGE = A_BYTES + B_BYTES;
    static constexpr int EPI_BYTES = 4 * 32 * 33 * 4;  // a padded 32 x 32 tile per drain warp
    static constexpr int FIT = (227 * 1024 - EPI_BYTES - 1024 - 256) / STAGE;
    static constexpr int STAGES = FIT > 8 ? 8 : FIT;
    static constexpr int SMEM_BYTES = STAGES * STAGE + EPI_BYTES + 1024 + 256;
    static constexpr int TMEM_COLS = 2 * BN;
    // D = FP32 (bits 4-5 = 1), A = B = FP16 (0), both K-major, N >> 3 at bit 17, M >> 4 at bit 24
    static constexpr uint32_t IDESC = (1u << 4) | ((uint32_t)(BN >> 3) << 17) | ((uint32_t)(BM >> 4) << 24);
    static_assert(BN == 64 || BN == 128 || BN == 256, "a power of two of tensor memory columns");
};

// D[tmem] (+)= A[smem desc] * B[smem desc]^T with FP16 inputs and FP32 accumulation.
__device__ __forceinline__ void umma_f16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Descriptor of a K-major operand in 128-byte swizzled rows (8 rows = 1024 bytes).
__device__ __forceinline__ uint64_t umma_desc_128b(uint32_t saddr) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)1u << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1u << 46) | ((uint64_t)2u << 61);
}

// Columns [c, c + n) of one output row from n FP32 sums.
template <int CT, int N>
__device__ __forceinline__ void store_outputs(void *C, int64_t at, const float *v) {
    if constexpr (CT == SGEMM_F32) {
        *reinterpret_cast<float4 *>(static_cast<float *>(C) + at) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
        *reinterpret_cast<uint4 *>(static_cast<typename Elem<CT>::type *>(C) + at) = pack16<CT>(v);
    }
}

// Units u = blockIdx.x, blockIdx.x + gridDim.x, ... of `splits` x tiles: tile
// u % tiles of the grouped raster, k-split u / tiles.  With splits > 1 each
// writes its raw sums to its own M x ldp slab of `partials` (CT is FP32 then),
// and i8_join_kernel adds the slabs in order and applies the scales.  debug: the
// test-only switches (bit 0: no copies, so that the waits run out).
template <int BN, int CT>
__global__ void __launch_bounds__(I8Tile<BN>::THREADS, 1)
    i8_tcgen05_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, const I8Args p,
                      int splits, float *__restrict__ partials, int64_t ldp, int vec, int *__restrict__ err_word,
                      unsigned long long wait_limit_ns, int debug) {
    using T = I8Tile<BN>;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    unsigned char *smem = smem_raw + (base - raw);
    // ring, staging tiles, then full[S], empty[S], acc_full[2], acc_empty[2], drained, flags
    const uint32_t bars = base + T::STAGES * T::STAGE + T::EPI_BYTES;
    const uint32_t full0 = bars, empty0 = bars + 8 * T::STAGES;
    const uint32_t acc_full0 = bars + 16 * T::STAGES, acc_empty0 = acc_full0 + 16, drained = acc_full0 + 32;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + (bars - base) + 16 * T::STAGES + 40);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + (bars - base) + 16 * T::STAGES + 44);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int tiles_m = (p.M + T::BM - 1) / T::BM, tiles_n = (p.N + BN - 1) / BN;
    const int tiles = tiles_m * tiles_n, units = tiles * splits;
    const int steps = (p.K + T::BK - 1) / T::BK;
    // unit u: output tile origin, first k-step and number of k-steps (at least one)
    auto unit = [&](int u, int &m0, int &n0, int &k0, int &n) {
        int tm, tn;
        grouped_tile<8>(u % tiles, tiles_m, tiles_n, tm, tn);
        m0 = tm * T::BM;
        n0 = tn * BN;
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
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
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
    // everything above may run beside the kernel that writes the operands
    griddep_wait();

    int issued = 0;  // copy thread: k-steps issued over all of this block's units
    if (warp == 0 && lane == 0) {
        prefetch_tensor_map(&tmA);
        prefetch_tensor_map(&tmB);
        for (int u = blockIdx.x; !(debug & 1) && u < units && !*abort_flag; u += gridDim.x) {
            int m0, n0, k0, n;
            unit(u, m0, n0, k0, n);
            for (int k = 0; k < n; ++k) {
                const int s = issued % T::STAGES, use = issued / T::STAGES;
                if (use > 0 && !mbar_wait_bounded(empty0 + 8 * s, (use - 1) & 1, wait_limit_ns)) *abort_flag = 1;
                if (*abort_flag) break;
                const uint32_t dst = base + s * T::STAGE, bar = full0 + 8 * s;
                mbar_arrive_expect_tx(bar, T::STAGE);
                tma_load_2d(dst, &tmA, (k0 + k) * T::BK, m0, bar);
                tma_load_2d(dst + T::A_BYTES, &tmB, (k0 + k) * T::BK, n0, bar);
                ++issued;
            }
        }
    } else if (warp == 1 && lane == 0) {
        int g = 0, i = 0;  // k-steps and units behind this block
        for (int u = blockIdx.x; u < units && !*abort_flag; u += gridDim.x, ++i) {
            int m0, n0, k0, n;
            unit(u, m0, n0, k0, n);
            const int b = i & 1, use = i >> 1;
            // the drain warps are done with this accumulator's previous tile
            if (use > 0 && !mbar_wait_bounded(acc_empty0 + 8 * b, (use - 1) & 1, wait_limit_ns)) {
                *abort_flag = 1;
                break;
            }
            tc_fence_after_sync();
            const uint32_t acc = tmem + (uint32_t)(b * BN);
            bool ok = true;
            for (int k = 0; k < n; ++k, ++g) {
                const int s = g % T::STAGES;
                if (!mbar_wait_bounded(full0 + 8 * s, (g / T::STAGES) & 1, wait_limit_ns)) {
                    *abort_flag = 1;
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                const uint32_t sa = base + s * T::STAGE, sb = sa + T::A_BYTES;
#pragma unroll
                for (int kk = 0; kk < T::BK / 16; ++kk)
                    umma_f16(acc, umma_desc_128b(sa + kk * 32), umma_desc_128b(sb + kk * 32), T::IDESC, (k | kk) != 0);
                umma_commit(empty0 + 8 * s);  // stage s may be refilled once these have read it
            }
            if (!ok) break;
            umma_commit(acc_full0 + 8 * b);  // the tile is final once its products are done
        }
        // every product issued above has completed before the block moves on
        umma_commit(drained);
        (void)mbar_wait_bounded(drained, 0, wait_limit_ns);
    } else if (warp >= 2) {
        // drain warps: lanes 32 q .. 32 q + 31 of a finished tile, 32 columns at a time through a
        // padded tile, so that the stores run along rows
        const int q = warp & 3;
        float *stage = reinterpret_cast<float *>(smem + T::STAGES * T::STAGE) + (warp - 2) * (32 * 33);
        constexpr int VEC = CT == SGEMM_F32 ? 4 : 8, LANES = 32 / VEC, ROWS = 32 / LANES;
        int i = 0;
        for (int u = blockIdx.x; u < units; u += gridDim.x, ++i) {
            int m0, n0, k0, n;
            unit(u, m0, n0, k0, n);
            const int b = i & 1;
            // a finished tile is stored whatever another role decided since
            const bool ready = mbar_wait_bounded(acc_full0 + 8 * b, (i >> 1) & 1, wait_limit_ns);
            if (!__all_sync(0xffffffffu, ready)) {
                if (lane == 0) *abort_flag = 1;
                break;
            }
            tc_fence_after_sync();
            const int row0 = m0 + 32 * q;
            const float row_scale = splits == 1 && row0 + lane < p.M ? p.a_scale[row0 + lane] : 1.f;
            void *out = splits > 1 ? static_cast<void *>(partials + (int64_t)(u / tiles) * p.M * ldp) : p.C;
            const int64_t ldo = splits > 1 ? ldp : p.ldc;
            const uint32_t acc = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(b * BN);
#pragma unroll 1
            for (int c0 = 0; c0 < BN; c0 += 32) {
                float v[32];
                tmem_ld32(acc + (uint32_t)c0, v);
                if (c0 + 32 == BN) {
                    // the accumulator is read: hand it back to the product thread
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(acc_empty0 + 8 * b);
                }
                if (n0 + c0 >= p.N || row0 >= p.M) continue;
#pragma unroll
                for (int j = 0; j < 32; ++j) stage[lane * 33 + j] = v[j] * row_scale;
                __syncwarp();
                const int col = n0 + c0;
                if (vec && col + 32 <= p.N) {
                    const int cq = (lane % LANES) * VEC, rr = lane / LANES;
                    float w[VEC], add[VEC];
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        w[e] = splits == 1 ? p.b_scale[col + cq + e] : 1.f;
                        add[e] = splits == 1 && p.bias ? p.bias[col + cq + e] : 0.f;
                    }
#pragma unroll
                    for (int r = rr; r < 32; r += ROWS) {
                        if (row0 + r < p.M) {
                            float o[VEC];
#pragma unroll
                            for (int e = 0; e < VEC; ++e) o[e] = fmaf(stage[r * 33 + cq + e], w[e], add[e]);
                            store_outputs<CT, VEC>(out, (int64_t)(row0 + r) * ldo + col + cq, o);
                        }
                    }
                } else if (col + lane < p.N) {
                    const float w = splits == 1 ? p.b_scale[col + lane] : 1.f;
                    const float add = splits == 1 && p.bias ? p.bias[col + lane] : 0.f;
#pragma unroll 8
                    for (int r = 0; r < 32; ++r)
                        if (row0 + r < p.M)
                            static_cast<typename Elem<CT>::type *>(out)[(int64_t)(row0 + r) * ldo + col + lane] =
                                Elem<CT>::from_float(fmaf(stage[r * 33 + lane], w, add));
                }
                __syncwarp();
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
            (void)mbar_wait_bounded(full0 + 8 * (t % T::STAGES), (t / T::STAGES) & 1, wait_limit_ns);
    }
    if (*abort_flag && splits > 1 && warp >= 2) {
        // this block's slabs are filled with NaN, so that no stale sums reach C
        for (int u = blockIdx.x; u < units; u += gridDim.x) {
            int m0, n0, k0, n;
            unit(u, m0, n0, k0, n);
            const int row = m0 + 32 * (warp & 3) + lane;
            if (row >= p.M) continue;
            for (int c = n0; c < min(n0 + BN, p.N); ++c)
                partials[(int64_t)(u / tiles) * p.M * ldp + row * ldp + c] = __int_as_float(0x7fc00000);
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 0) tmem_dealloc(tmem, T::TMEM_COLS);
}

// Adds the k-splits' slabs in order and applies the scales and the bias.
__global__ void __launch_bounds__(256) i8_join_kernel(const I8Args p, int splits, const float *__restrict__ partials,
                                                      int64_t ldp) {
    const int64_t total = (int64_t)p.M * p.N, slab = (int64_t)p.M * ldp;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t m = i / p.N;
        const int n = (int)(i - m * p.N);
        const float *at = partials + (splits > 0 ? m * ldp + n : 0);
        float s = splits > 0 ? at[0] : 0.f;  // no k at all: an empty sum
        for (int k = 1; k < splits; ++k) s += at[k * slab];
        s *= p.a_scale[m];
        store_c(p.C, m * p.ldc + n, p.ctype, fmaf(s, p.b_scale[n], p.bias ? p.bias[n] : 0.f));
    }
}

}  // namespace sgemm
