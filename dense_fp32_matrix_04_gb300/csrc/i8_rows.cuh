// The product of 8-bit operands for up to four tokens: the time is that of
// reading B, N K bytes, once.
//
// A warp takes a row of B at a time and reads it in pieces of 512 contiguous
// bytes, eight in flight a lane; with four-way byte products into 32-bit
// integers (exact) it spends 4 M + 1 instructions on 16 bytes a lane, so the
// loads, not the arithmetic, set the pace.  The tokens' codes stay in shared
// memory; where the tokens come unquantised, every block quantises them itself
// (M K elements from L2) while its first row of B is on its way, which saves a
// kernel of its own in front.
//
// One token by 4096 x 4096 takes 4.9 - 5.2 us (3.4 TB/s of B): 2.5 are B's bytes,
// the rest a launch, the quantised row and the last loads' latency.  From five
// tokens on the byte products, 273 a cycle and SM, would set the pace, and the
// tensor cores are faster (i8_stream.cuh; 11.4 us there for five tokens).
//
// The sums are exact for every K, so long rows stay here: four tokens' codes fit
// shared memory up to K = 57344 (4 x 5120 x 28672 42.4 us, 50.9 for five tokens on
// the tensor cores; with codes that come quantised 39.4 and 34.9); beyond, two or
// one at a time read B once for each (4 x 4096 x 65536 130 us, 92 for five).
#pragma once

#include <cstdint>

#include "i8_codes.cuh"
#include "i8_quantize.cuh"

namespace sgemm {

constexpr int kRowsTokens = 4;
constexpr int kRowsThreads = 256, kRowsWideThreads = 768;  // a block's; see kRowsWide
constexpr int kRowsPieces = 8;  // loads of 16 bytes a lane has in flight

constexpr int kRowsCodes = 224 * 1024;  // shared memory that a block's tokens' codes may take
// Codes of more than this leave room for too few blocks of 256 threads, and so for
// too few loads on their way: one block of 768 then (4 x 5120 x 28672 53.9 -> 42.4
// us, 2 x 5120 x 28672 37.6 -> 32.1, 4 x 4096 x 14336 23.5 and 23.8).
constexpr int kRowsWide = 52 * 1024;

// Bytes of a token's codes in shared memory: whole rounds of loads.
__host__ __device__ constexpr int rows_pitch(int K) { return (K + 511) / 512 * 512; }

// XT: the tokens are codes (-1) or values of that element type.
template <int MT, int XT, bool ALIGNED, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS > kRowsThreads ? 1 : MT < 4 && ALIGNED ? 4 : 3)
    i8_rows_kernel(const I8Args p, const void *__restrict__ X, int64_t ldx) {
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ float slots[THREADS / 32], scales[MT];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, K = p.K;
    const int pitch = rows_pitch(K);
    const int warps = gridDim.x * (THREADS / 32);
    int row = blockIdx.x * (THREADS / 32) + warp;

    auto load = [&](uint4 (&w)[kRowsPieces], const int8_t *from, int k0) {
#pragma unroll
        for (int j = 0; j < kRowsPieces; ++j) w[j] = load_codes<ALIGNED>(from, k0 + 512 * j + 16 * lane, K);
    };
    uint4 w[kRowsPieces];
    const int8_t *from = p.B + (int64_t)min(row, p.N - 1) * p.ldb;
    load(w, from, 0);

    if constexpr (XT < 0) {
        // 16 codes at a time; those past the row's end are 0
        for (int m = 0; m < MT; ++m)
#pragma unroll 4
            for (int k = 16 * tid; k < pitch; k += 16 * THREADS) {
                const uint4 c = load_codes<false>(p.A + m * p.lda, k, m < p.M ? K : 0);
                uint32_t word[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int left = K - k - 4 * i;
                    word[i] = left >= 4 ? word[i] : left > 0 ? word[i] & ((1u << 8 * left) - 1) : 0u;
                }
                *reinterpret_cast<uint4 *>(smem + m * pitch + k) = make_uint4(word[0], word[1], word[2], word[3]);
            }
        if (tid < MT) scales[tid] = tid < p.M ? p.a_scale[tid] : 0.f;
    } else {
        // the block's warps are shared out to the tokens, which are quantised side by side
        using E = Elem<XT < 0 ? 0 : XT>;
        constexpr int SHARE = THREADS / 32 / MT, VEC = E::VEC;
        const int m = warp / SHARE, first = (warp % SHARE) * 32 + lane, step = SHARE * 32;
        const typename E::type *x = static_cast<const typename E::type *>(X) + min(m, p.M - 1) * ldx;
        const int pieces = (reinterpret_cast<uintptr_t>(x) & 15) == 0 ? K / VEC : 0;
        uint32_t top = 0;
        auto larger = [&](float v) { top = max(top, __float_as_uint(v) & 0x7fffffffu); };
#pragma unroll 4
        for (int i = first; i < pieces; i += step) {
            float v[VEC];
            unpack16<(XT < 0 ? 0 : XT)>(__ldg(reinterpret_cast<const uint4 *>(x) + i), v);
#pragma unroll
            for (int e = 0; e < VEC; ++e) larger(v[e]);
        }
#pragma unroll 4
        for (int k = pieces * VEC + first; k < K; k += step) larger(E::to_float(x[k]));
        top = warp_max(top);
        if (lane == 0) slots[warp] = __uint_as_float(top);
        __syncthreads();
        for (int i = 0; i < SHARE; ++i) top = max(top, __float_as_uint(slots[m * SHARE + i]));
        const I8Scale s(top);
        unsigned char *codes = smem + m * pitch;
#pragma unroll 4
        for (int i = first; i < pieces; i += step) {
            float v[VEC];
            unpack16<(XT < 0 ? 0 : XT)>(__ldg(reinterpret_cast<const uint4 *>(x) + i), v);
            int8_t c[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) c[e] = s(v[e]);
            store_bytes(reinterpret_cast<int8_t *>(codes) + i * VEC, c, true);
        }
#pragma unroll 4
        for (int k = pieces * VEC + first; k < pitch; k += step)
            codes[k] = k < K ? (unsigned char)s(E::to_float(x[k])) : 0;
        if (warp % SHARE == 0 && lane == 0) scales[m] = s.scale;
    }
    __syncthreads();

    for (; row < p.N; row += warps) {
        int acc[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[m] = 0;
        for (int k0 = 0; k0 < K; k0 += 512 * kRowsPieces) {
            if (k0 > 0) load(w, from, k0);
#pragma unroll
            for (int j = 0; j < kRowsPieces; ++j) {
                const int k = k0 + 512 * j;
                if (k >= K) break;
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    // codes past the row's end are 0, whatever the piece of B holds there
                    const uint4 x = *reinterpret_cast<const uint4 *>(smem + m * pitch + k + 16 * lane);
                    acc[m] = __dp4a((int)w[j].x, (int)x.x, acc[m]);
                    acc[m] = __dp4a((int)w[j].y, (int)x.y, acc[m]);
                    acc[m] = __dp4a((int)w[j].z, (int)x.z, acc[m]);
                    acc[m] = __dp4a((int)w[j].w, (int)x.w, acc[m]);
                }
            }
        }
        const int next = row + warps;
        from = p.B + (int64_t)min(next, p.N - 1) * p.ldb;
        if (next < p.N) load(w, from, 0);
        int mine = 0;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int sum = __reduce_add_sync(0xffffffffu, acc[m]);
            if (lane == m) mine = sum;
        }
        if (lane < MT && lane < p.M)
            store_c(p.C, lane * p.ldc + row, p.ctype,
                    fmaf((float)mine * scales[lane], p.b_scale[row], p.bias ? p.bias[row] : 0.f));
    }
}

}  // namespace sgemm
