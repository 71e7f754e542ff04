// The norm of rows about their mean, after the sum of the residual stream and a
// block's output, and its gradient:
//     r = x + a                       (rounded to the rows' type, and handed on)
//     n = (r - mean) rstd w + b,      rstd = rsqrt(mean((r - mean)^2) + eps)
// What is normalised is the r that is handed on, so that the gradient needs r alone.
// A row is read once into registers and walked as in block_norm.cuh; its two moments
// are each warp's own, about its own mean, joined with one barrier.
//
// Memory bounds both: 8192 x 5120 BF16 with a sum and a bias takes 61.5 us, 5.5 TB/s, the
// gradient of 8192 x 4096 with one from r 48.3 us, 5.6 TB/s (without 39.1), 2 of them
// joining the blocks' sums.  (Inputs in turn over more than L2 holds, here and below unless said
// otherwise.)  (Clusters of two or four blocks that add theirs first: the same, and 40 %
// slower, as fours leave SMs without a block.  L2 fetches of 128 and 256 bytes: the same.)
// Rows of a cluster of blocks, beyond 8192 columns (FP32 with a sum: 7168), are bound by its barriers,
// two a row one after the other with nothing else on the SM: 501 x 22224 BF16 76 us forward and 65
// backward, 2000 x 8192 FP32 87, where memory needs 13 and 39.
// Rows that are not whole 16 bytes are read and written as single elements and
// take 1.0 (FP32 forward) to 2 times as long: 4000 x 5119 BF16 50 us, x 5120 30.  (Whole
// pieces of them, shifted in registers and handed on to the neighbouring lane, took three
// times the instructions: forward 7 % slower, the gradient 10 % faster; not kept.)
#pragma once

#include <cstdint>

#include "ptx.cuh"
#include "row_ring.cuh"
#include "rows.cuh"

namespace sgemm {

struct LayerNormArgs {
    int T, D;
    const void *x, *add;
    int64_t ldx, lda;
    const void *w, *b;
    int w_f32;         // the weights are FP32 (otherwise of the rows' type)
    float eps;
    void *r, *n;
    int64_t ldr, ldn;
    float *stats;      // 2 x T: mean, rstd
    int ranks, width;  // blocks that share a row, and the columns of each
};

struct LayerNormGradArgs {
    int T, D;
    const void *x, *dn, *dr;
    int64_t ldx, lddn, lddr;
    const void *w;
    int w_f32;
    const float *stats;
    void *dx;
    int64_t lddx;
    void *dw, *db;
    float *partial;    // partials x 2 x D: dw, db
    int runners;       // of the rows: blocks (or clusters), or for narrow rows the four warps of each
    int partials;      // blocks (or clusters)
    int ranks, width;
};

constexpr int kLayerNormStages = 4;
constexpr int kLayerNormGradStages = 3;

// The threads of a row: as in block_norm_kernel.
template <int DT, bool ALIGNED, int NV, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) layer_norm_kernel(const LayerNormArgs a) {
    using L = RowLayout<DT, ALIGNED, NV>;
    using type = typename L::type;
    constexpr int V = L::VEC, H = V / 2, S = kLayerNormStages;  // H pairs a piece
    extern __shared__ uint4 ring[];
    __shared__ float slots[RowReducer::SLOTS];
    RowReducer red{slots, (int)(blockDim.x >> 5), a.ranks};
    const int rank = (int)(blockIdx.x % (unsigned)a.ranks), group_id = (int)(blockIdx.x / (unsigned)a.ranks);
    const int c0 = rank * a.width;  // this block's columns
    const L l(min(a.width, a.D - c0));
    const int cols = c0 + l.col;
    const float inv_d = 1.f / (float)a.D;
    const int arrays = a.add ? 2 : 1, pieces = l.pieces();
    uint4 *mine = l.place(ring, S * arrays);

    F2 w[NV][H], b[NV][H];
    const int wsize = a.w_f32 ? 4 : (int)sizeof(type);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        l.template weights<V>(static_cast<const char *>(a.w) + (int64_t)c0 * wsize, a.w_f32, v * V, w[v]);
        if (a.b) {
            l.template weights<V>(static_cast<const char *>(a.b) + (int64_t)c0 * wsize, a.w_f32, v * V, b[v]);
        } else {
#pragma unroll
            for (int i = 0; i < H; ++i) b[v][i] = F2(0.f);
        }
    }
    const float count = l.warp_columns(), inv_count = count > 0.f ? 1.f / count : 0.f;

    const int64_t first = (int64_t)group_id * blockDim.y + threadIdx.y;
    const int64_t step = (int64_t)(gridDim.x / (unsigned)a.ranks) * blockDim.y;
    // rows are numbered below 2^30 and leading dimensions are 32-bit: one multiplication
    auto row = [&](const void *p, int64_t ld, int64_t t) {
        return static_cast<const type *>(p) + ((int64_t)(int)t * (int)ld + cols);
    };
    auto fetch = [&](int64_t t, int stage) {
        if (t < a.T) {
            uint4 *slot = mine + stage * arrays * pieces;
            l.copy(slot, row(a.x, a.ldx, t));
            if (a.add) l.copy(slot + pieces, row(a.add, a.lda, t));
        }
        cp_async_commit();
    };
#pragma unroll
    for (int s = 0; s < S - 1; ++s) fetch(first + s * step, s);

    int stage = 0;
    for (int64_t t = first; t < a.T; t += step) {
        cp_async_wait<S - 2>();
        if (!ALIGNED) row_sync(red.warps);
        const uint4 *slot = mine + stage * arrays * pieces;
        F2 r[NV][H], sum(0.f), square(0.f);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            l.template read<V>(slot, row(a.x, a.ldx, t), v * V, r[v]);
            if (a.add) {
                F2 y[H];
                l.template read<V>(slot + pieces, row(a.add, a.lda, t), v * V, y);
#pragma unroll
                for (int i = 0; i < H; ++i) r[v][i] = r[v][i] + y[i];
                l.store(const_cast<type *>(row(a.r, a.ldr, t)), v * V, r[v]);
                L::rounded(r[v]);
            }
#pragma unroll
            for (int i = 0; i < H; ++i) sum = sum + r[v][i];
        }
        // the slot that the previous row was read from takes the row after the next ones
        fetch(t + (S - 1) * step, stage == 0 ? S - 1 : stage - 1);
        stage = stage == S - 1 ? 0 : stage + 1;
        float mean, var;
        // sum of squares about `about`, of this thread's columns
        auto squares = [&](float about) {
            F2 ss(0.f);
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    F2 d = r[v][i] + F2(-about);
                    l.only_inside(v * V + 2 * i, d);
                    ss = fma(d, d, ss);
                }
            return ss.sum();
        };
        if (a.ranks > 1) {
            mean = red.sum(sum.sum()) * inv_d;
            var = red.sum(squares(mean)) * inv_d;
        } else {
            const float s = warp_sum(sum.sum());
            red.moments(count, s, warp_sum(squares(s * inv_count)), inv_d, mean, var);
        }
        const float rstd = rsqrtf(var + a.eps);
        if (a.stats && threadIdx.x == 0 && rank == 0) {
            a.stats[t] = mean;
            a.stats[a.T + t] = rstd;
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
#pragma unroll
            for (int i = 0; i < H; ++i) r[v][i] = fma((r[v][i] + F2(-mean)) * F2(rstd), w[v][i], b[v][i]);
            l.store(const_cast<type *>(row(a.n, a.ldn, t)), v * V, r[v]);
        }
    }
    if (a.ranks > 1) cluster_sync();
}

// With h = (x - mean) rstd and u = dn w the gradient of a row is
//     dx = dr + rstd (u - mean(u) - h mean(u h)),
// two sums, taken at once, so a row costs one barrier.  dw = sum dn h and db = sum dn
// over a runner's rows stay in registers; what a block has of them (of narrow rows its four
// warps, added in shared memory: 16000 x 512 BF16 in L2 12.4 us, 18.9 without) goes to `partial`, where a
// second kernel adds the blocks in order.
template <int DT, bool ALIGNED, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT, 1) layer_norm_grad_kernel(const LayerNormGradArgs a) {
    using L = RowLayout<DT, ALIGNED, NV>;
    using type = typename L::type;
    constexpr int N = L::N, V = L::VEC, P = V / 2, S = kLayerNormGradStages;  // P pairs a piece
    extern __shared__ uint4 ring[];
    __shared__ float slots[RowReducer::SLOTS];
    griddep_launch_dependents();  // the kernel that joins the runners' sums, which waits for this one
    RowReducer red{slots, (int)(blockDim.x >> 5), a.ranks};
    const int rank = (int)(blockIdx.x % (unsigned)a.ranks), group_id = (int)(blockIdx.x / (unsigned)a.ranks);
    const int c0 = rank * a.width;  // this block's columns
    const L l(min(a.width, a.D - c0));
    const int cols = c0 + l.col;
    const float inv_d = 1.f / (float)a.D;
    const int runner = group_id * blockDim.y + threadIdx.y;
    const RowRuns runs(a.T, a.runners);
    const bool idle = runner >= a.runners;  // only where a warp is a runner
    const int begin = idle ? 0 : runs.first(runner), end = idle ? 0 : runs.first(runner + 1);
    const int arrays = a.dr ? 3 : 2, pieces = l.pieces(), stride = arrays * pieces;
    uint4 *mine = l.place(ring, S * arrays);

    F2 w[N / 2], dw[N / 2], db[N / 2];
    const int wsize = a.w_f32 ? 4 : (int)sizeof(type);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        F2 f[P];
        l.template weights<V>(static_cast<const char *>(a.w) + (int64_t)c0 * wsize, a.w_f32, v * V, f);
#pragma unroll
        for (int i = 0; i < P; ++i) w[v * P + i] = f[i];
    }
#pragma unroll
    for (int i = 0; i < N / 2; ++i) dw[i] = db[i] = F2(0.f);

    auto at = [&](const void *p, int64_t ld, int t) { return static_cast<const type *>(p) + ((int64_t)t * (int)ld + cols); };
    auto fetch = [&](int t, int stage) {
        if (t < end) {
            uint4 *slot = mine + stage * stride;
            l.copy(slot, at(a.x, a.ldx, t));
            l.copy(slot + pieces, at(a.dn, a.lddn, t));
            if (a.dr) l.copy(slot + 2 * pieces, at(a.dr, a.lddr, t));
        }
        cp_async_commit();
    };
#pragma unroll
    for (int k = 0; k < S - 1; ++k) fetch(begin + k, k);

    int stage = 0;
    for (int t = begin; t < end; ++t) {
        cp_async_wait<S - 2>();
        if (!ALIGNED) row_sync(red.warps);
        const uint4 *slot = mine + stage * stride;
        fetch(t + S - 1, stage == 0 ? S - 1 : stage - 1);
        stage = stage == S - 1 ? 0 : stage + 1;
        const float mean = a.stats[t], rstd = a.stats[a.T + t];
        F2 h[N / 2], u[N / 2], part[2] = {F2(0.f), F2(0.f)};
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            F2 xx[P], d[P];
            l.template read<V>(slot, at(a.x, a.ldx, t), v * V, xx);
            l.template read<V>(slot + pieces, at(a.dn, a.lddn, t), v * V, d);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                // (past the row's end dn is 0)
                const int k = v * P + i;
                h[k] = (xx[i] + F2(-mean)) * F2(rstd);
                dw[k] = fma(d[i], h[k], dw[k]);
                db[k] = db[k] + d[i];
                u[k] = d[i] * w[k];
                part[0] = part[0] + u[k];
                part[1] = fma(u[k], h[k], part[1]);
            }
        }
        float sums[2] = {part[0].sum(), part[1].sum()};
        red.sum(sums);
        const float c1 = sums[0] * inv_d * rstd, c2 = sums[1] * inv_d * rstd;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            F2 d[P];
            if (a.dr) {
                l.template read<V>(slot + 2 * pieces, at(a.dr, a.lddr, t), v * V, d);
            } else {
#pragma unroll
                for (int i = 0; i < P; ++i) d[i] = F2(0.f);
            }
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int k = v * P + i;
                d[i] = d[i] + fma(h[k], F2(-c2), fma(u[k], F2(rstd), F2(-c1)));
            }
            l.store(static_cast<type *>(a.dx) + ((int64_t)t * (int)a.lddx + cols), v * V, d);
        }
    }
    // (a.D is no more than NV pieces of a warp where a block has several runners)
    const bool shared = blockDim.y > 1;
    float *sums = shared ? reinterpret_cast<float *>(ring) + threadIdx.y * 2 * a.D : a.partial + (int64_t)group_id * 2 * a.D;
    if (shared) {
        cp_async_wait<0>();
        __syncthreads();  // nobody's rows are on their way, or read, any more
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        l.put(sums + cols, v * V, dw + v * P, false);
        if (a.db) l.put(sums + a.D + cols, v * V, db + v * P, false);
    }
    if (shared) {
        __syncthreads();
        const int n = (a.db ? 2 : 1) * a.D;
        for (int i = threadIdx.y * 32 + threadIdx.x; i < n; i += 32 * blockDim.y) {
            const float *from = reinterpret_cast<const float *>(ring) + i;
            float sum = from[0];
            for (int y = 1; y < (int)blockDim.y; ++y) sum += from[y * 2 * a.D];
            a.partial[(int64_t)group_id * 2 * a.D + i] = sum;
        }
    }
    if (a.ranks > 1) cluster_sync();
}

// Adds the blocks' partial sums, blockIdx.y 0 of dw and 1 of db: 32 columns by
// kLayerNormJoinSlices slices of the blocks, each added in order with LOADS loads on
// their way, then the slices in order.  (With an address computed in 64 bits for each load the
// kernel took 600 instructions a warp, and the gradient of 300 x 4096, in L2, 12.4 us instead of 8.6.)
constexpr int kLayerNormJoinSlices = 16;
template <int DT>
__global__ void __launch_bounds__(32 * kLayerNormJoinSlices) layer_norm_grad_join_kernel(const LayerNormGradArgs a) {
    constexpr int LOADS = 20, SLICES = kLayerNormJoinSlices;
    __shared__ float part[SLICES][32];
    const int c = blockIdx.x * 32 + threadIdx.x, k = blockIdx.y;
    griddep_wait();
    float s = 0.f;
    if (c < a.D)
        for (int b = threadIdx.y; b < a.partials; b += LOADS * SLICES) {
            // (the sums of all blocks are a few million at most)
            const float *from = a.partial + (b * 2 + k) * a.D + c;
            float v[LOADS];
#pragma unroll
            for (int i = 0; i < LOADS; ++i, from += SLICES * 2 * a.D) v[i] = b + i * SLICES < a.partials ? __ldcg(from) : 0.f;
#pragma unroll
            for (int i = 0; i < LOADS; ++i) s += v[i];
        }
    part[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < a.D) {
#pragma unroll
        for (int i = 1; i < SLICES; ++i) s += part[i][threadIdx.x];
        store_weight<DT>(k ? a.db : a.dw, a.w_f32, c, s);
    }
}

}  // namespace sgemm
