// The norms, gate and residual sum between two blocks of a model, and their
// gradient:
//     h = y rho w_post,  rho = rsqrt(mean(y^2) + eps)
//     r = x + a g h
//     n = r rho2 w_pre,  rho2 = rsqrt(mean(r^2) + eps)
// A row is read once into registers, its two sums of squares are reduced over
// the threads that share it, and r and n are written once.  At about ten
// operations an element the kernels are bound by memory.
#pragma once

#include <cstdint>

#include "i8_quantize.cuh"
#include "ptx.cuh"
#include "rows.cuh"

namespace sgemm {

struct BlockNormArgs {
    int T, D;
    const void *x, *y, *gate;
    int64_t ldx, ldy, ldg;
    const void *w_pre, *w_post;
    int w_f32;         // the weights are FP32 (otherwise of the rows' type)
    int gate_period;   // rows per gate row; 0: no gate
    float scale, eps;
    void *r, *n;
    int64_t ldr, ldn;
    int8_t *q;
    int64_t ldq;
    float *q_scale;
    float *rstd;
    int q_vec;         // rows of q allow stores of a whole piece
    int ranks, width;  // blocks that share a row, and the columns of each
};

struct BlockNormGradArgs {
    int T, D;
    const void *x, *y, *gate, *dn, *dr;
    int64_t ldx, ldy, ldg, lddn, lddr;
    const void *w_pre, *w_post;
    int w_f32;
    int gate_period;
    float scale;
    const float *rstd;
    void *dx, *dy, *dgate;
    int64_t lddx, lddy, lddg;
    void *dw_pre, *dw_post;
    float *partial;    // runners x 4 x D: dw_pre, dw_post, and the gate rows a runner has a part of
    int runners;
    int ranks, width;  // as above
};

template <int DT>
__device__ __forceinline__ float load_weight(const void *w, int w_f32, int c) {
    using E = Elem<DT>;
    return w_f32 ? static_cast<const float *>(w)[c] : E::to_float(static_cast<const typename E::type *>(w)[c]);
}

template <int DT>
__device__ __forceinline__ void store_weight(void *w, int w_f32, int64_t c, float v) {
    using E = Elem<DT>;
    if (w_f32) static_cast<float *>(w)[c] = v;
    else static_cast<typename E::type *>(w)[c] = E::from_float(v);
}

// ---------------------------------------------------------------- rows through shared memory
//
// The threads that share a row copy the next rows' inputs into shared memory
// (cp.async, whole 16-byte pieces) while they work on this one, so what is in
// flight does not depend on how many blocks fit an SM.  With ALIGNED rows
// (16-byte aligned and a whole number of pieces) each thread copies the pieces
// it will read itself and needs no barrier; any other row is copied as the
// pieces that enclose it (up to 15 bytes in front and behind are read and
// never used), a barrier lets the row's threads see each other's copies, and
// they read single elements.
template <int DT, bool ALIGNED, int NV>
struct RowLayout {
    using type = typename Elem<DT>::type;
    static constexpr int VEC = Elem<DT>::VEC, N = NV * VEC;  // elements a thread
    // column of this thread's element i
    __device__ static int col(int i, int threads, int tx) {
        return ALIGNED ? ((i / VEC) * threads + tx) * VEC + i % VEC : i * threads + tx;
    }
    // starts the copies of a row into `slot`
    __device__ static void copy(uint4 *slot, const type *row, int D, int threads, int tx) {
        if constexpr (ALIGNED) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int p = v * threads + tx;
                if (p * VEC < D) cp_async_16(smem_addr(slot + p), row + p * VEC, 16);
            }
        } else {
            const uintptr_t lo = reinterpret_cast<uintptr_t>(row) & ~(uintptr_t)15;
            const int pieces = (int)((reinterpret_cast<uintptr_t>(row + D) + 15 - lo) >> 4);
            for (int p = tx; p < pieces; p += threads)
                cp_async_16(smem_addr(slot + p), reinterpret_cast<const void *>(lo + 16 * (uintptr_t)p), 16);
        }
    }
    // this thread's elements of the row that was copied from `row`; 0 past its end
    __device__ static void read(const uint4 *slot, const type *row, int D, int threads, int tx, float *out) {
        if constexpr (ALIGNED) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int p = v * threads + tx;
                unpack16<DT>(p * VEC < D ? slot[p] : make_uint4(0, 0, 0, 0), out + v * VEC);
            }
        } else {
            const type *e = reinterpret_cast<const type *>(slot) + (reinterpret_cast<uintptr_t>(row) & 15) / sizeof(type);
#pragma unroll
            for (int i = 0; i < N; ++i) out[i] = i * threads + tx < D ? Elem<DT>::to_float(e[i * threads + tx]) : 0.f;
        }
    }
    __device__ static void store(type *row, int D, int threads, int tx, const float *v) {
        if constexpr (ALIGNED) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int p = k * threads + tx;
                if (p * VEC < D) *reinterpret_cast<uint4 *>(row + p * VEC) = pack16<DT>(v + k * VEC);
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (i * threads + tx < D) row[i * threads + tx] = Elem<DT>::from_float(v[i]);
        }
    }
    // the same, two elements to a register pair
    __device__ static void read(const uint4 *slot, const type *row, int D, int threads, int tx, F2 *out) {
        float v[N];
        read(slot, row, D, threads, tx, v);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) out[i] = F2(v[2 * i], v[2 * i + 1]);
    }
    __device__ static void store(type *row, int D, int threads, int tx, const F2 *v) {
        float f[N];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float2 b = v[i].both();
            f[2 * i] = b.x;
            f[2 * i + 1] = b.y;
        }
        store(row, D, threads, tx, f);
    }
    __device__ static void weights(const void *w, int w_f32, int c0, int D, int threads, int tx, F2 *out) {
        float v[N];
        weights(w, w_f32, c0, D, threads, tx, v);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) out[i] = F2(v[2 * i], v[2 * i + 1]);
    }
    // 0 past the row's end; ALIGNED weights start on 16 bytes
    __device__ static void weights(const void *w, int w_f32, int c0, int D, int threads, int tx, float *out) {
        if constexpr (ALIGNED) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int c = (v * threads + tx) * VEC;
                if (c >= D) {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) out[v * VEC + e] = 0.f;
                } else if (w_f32) {
#pragma unroll
                    for (int e = 0; e < VEC; e += 4) {
                        const float4 q = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(w) + c0 + c + e));
                        out[v * VEC + e] = q.x, out[v * VEC + e + 1] = q.y;
                        out[v * VEC + e + 2] = q.z, out[v * VEC + e + 3] = q.w;
                    }
                } else {
                    unpack16<DT>(__ldg(reinterpret_cast<const uint4 *>(static_cast<const type *>(w) + c0 + c)), out + v * VEC);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                out[i] = i * threads + tx < D ? load_weight<DT>(w, w_f32, c0 + i * threads + tx) : 0.f;
        }
    }
};

// Rows a thread keeps on their way (and the one it works on).
constexpr int kNormStages = 4;
constexpr int kNormGradStages = 3;

// Copies of the inputs of one row, by the threads that share it.
__host__ __device__ constexpr int row_pieces(int D, int size) { return (D * size + 15) / 16 + 1; }

// The barrier of the threads that share a row.
__device__ __forceinline__ void row_sync(int warps) {
    if (warps == 1) __syncwarp();
    else __syncthreads();
}

// The threads of a row: blockDim.x of a block (and blockDim.y rows side by
// side in it, more than one only where a warp is enough for a row), in each of
// the `ranks` blocks of a cluster, which take `width` columns each.
template <int DT, bool ALIGNED, int NV, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) block_norm_kernel(const BlockNormArgs a) {
    using L = RowLayout<DT, ALIGNED, NV>;
    using type = typename L::type;
    constexpr int N = L::N, S = kNormStages;
    extern __shared__ uint4 ring[];
    __shared__ float slots[RowReducer::SLOTS];
    RowReducer red{slots, (int)(blockDim.x >> 5), a.ranks};
    const int threads = blockDim.x, tx = threadIdx.x;
    const int rank = (int)(blockIdx.x % (unsigned)a.ranks), group_id = (int)(blockIdx.x / (unsigned)a.ranks);
    const int c0 = rank * a.width, D = min(a.width, a.D - c0);  // this block's columns
    const float inv_d = 1.f / (float)a.D;
    const bool token_gate = a.gate_period == 1;
    const int arrays = token_gate ? 3 : 2, pieces = row_pieces(a.width, sizeof(type));
    uint4 *mine = ring + threadIdx.y * S * arrays * pieces;

    float w_pre[N], w_post[N];
    L::weights(a.w_pre, a.w_f32, c0, D, threads, tx, w_pre);
    if (a.w_post) L::weights(a.w_post, a.w_f32, c0, D, threads, tx, w_post);

    const int64_t first = (int64_t)group_id * blockDim.y + threadIdx.y;
    const int64_t step = (int64_t)(gridDim.x / (unsigned)a.ranks) * blockDim.y;
    auto x_row = [&](int64_t t) { return static_cast<const type *>(a.x) + t * a.ldx + c0; };
    auto y_row = [&](int64_t t) { return static_cast<const type *>(a.y) + t * a.ldy + c0; };
    auto g_row = [&](int64_t t) { return static_cast<const type *>(a.gate) + (int64_t)((unsigned)t / (unsigned)a.gate_period) * a.ldg + c0; };
    auto fetch = [&](int64_t t, int stage) {
        if (t < a.T) {
            uint4 *slot = mine + stage * arrays * pieces;
            L::copy(slot, x_row(t), D, threads, tx);
            L::copy(slot + pieces, y_row(t), D, threads, tx);
            if (token_gate) L::copy(slot + 2 * pieces, g_row(t), D, threads, tx);
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
        float h[N], r[N];
        L::read(slot + pieces, y_row(t), D, threads, tx, h);
        L::read(slot, x_row(t), D, threads, tx, r);
        float rho = 1.f;
        if (a.w_post) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < N; ++i) ss = fmaf(h[i], h[i], ss);
            rho = rsqrtf(fmaf(red.sum(ss), inv_d, a.eps));
#pragma unroll
            for (int i = 0; i < N; ++i) h[i] *= rho * w_post[i];
        }
        if (a.gate_period) {
            float g[N];
            if (token_gate) {
                L::read(slot + 2 * pieces, g_row(t), D, threads, tx, g);
            } else if constexpr (ALIGNED) {
                const type *row = g_row(t);  // the same for many rows: from L1
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    const int c = (v * threads + tx) * L::VEC;
                    unpack16<DT>(c < D ? __ldg(reinterpret_cast<const uint4 *>(row + c)) : make_uint4(0, 0, 0, 0),
                                 g + v * L::VEC);
                }
            } else {
                const type *row = g_row(t);
#pragma unroll
                for (int i = 0; i < N; ++i)
                    g[i] = i * threads + tx < D ? Elem<DT>::to_float(row[i * threads + tx]) : 0.f;
            }
#pragma unroll
            for (int i = 0; i < N; ++i) h[i] *= g[i];
        }
        // the slot that the previous row was read from takes the row after the next ones
        fetch(t + (S - 1) * step, stage == 0 ? S - 1 : stage - 1);
        stage = stage == S - 1 ? 0 : stage + 1;
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            r[i] = fmaf(a.scale, h[i], r[i]);
            ss = fmaf(r[i], r[i], ss);
        }
        L::store(static_cast<type *>(a.r) + t * a.ldr + c0, D, threads, tx, r);
        const float rho2 = rsqrtf(fmaf(red.sum(ss), inv_d, a.eps));
        if (a.rstd && tx == 0 && rank == 0) {
            a.rstd[t] = rho;
            a.rstd[a.T + t] = rho2;
        }
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            r[i] *= rho2 * w_pre[i];
            top = max(top, __float_as_uint(r[i]) & 0x7fffffffu);
        }
        if (a.n) L::store(static_cast<type *>(a.n) + t * a.ldn + c0, D, threads, tx, r);
        if (a.q) {
            const I8Scale q(red.max(top));
            if (tx == 0 && rank == 0) a.q_scale[t] = q.scale;
            int8_t *out = a.q + t * a.ldq + c0;
            if constexpr (ALIGNED) {
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    const int c = (v * threads + tx) * L::VEC;
                    if (c >= D) continue;
                    int8_t b[L::VEC];
#pragma unroll
                    for (int e = 0; e < L::VEC; ++e) b[e] = q(r[v * L::VEC + e]);
                    store_bytes(out + c, b, a.q_vec);
                }
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (i * threads + tx < D) out[i * threads + tx] = q(r[i]);
            }
        }
    }
    if (a.ranks > 1) cluster_sync();
}

// ---------------------------------------------------------------- gradient

// Runner b (a block, or a warp of one) takes consecutive rows, so that a gate
// row's sum stays in registers until the row changes: T / runners of them, and
// the first T % runners runners one more.  No division of 64 bits is on the way
// of a row (each cost about 100 instructions).
struct RowRuns {
    int each, more;
    __device__ RowRuns(int T, int runners) : each(T / runners), more(T % runners) {}
    __device__ int first(int b) const { return b * each + min(b, more); }
    __device__ int runner_of(int t) const {
        const int wide = more * (each + 1);
        return t < wide ? t / (each + 1) : more + (t - wide) / each;
    }
};

// The gradient of a row needs, with u = dn w_pre and v = dh w_post,
//     dx = dr + rho2 (u - r rho2^2 mean(u r)),   dh = a g dx,
//     dy = rho (v - y rho^2 mean(v y)),
// with rho and rho2 from the forward pass.  The second mean need not wait for
// the first: with P = a g w_post rho y,
//     sum(v rho y) = sum(P (dr + rho2 u)) - rho2^3 mean(u r) sum(P r),
// so three sums are taken at once, and a row costs one barrier.  Sums over rows (weights and gate) are kept in registers, and
// written per runner to `partial`: a second kernel adds the runners in order.
template <int DT, bool ALIGNED, int NV, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) block_norm_grad_kernel(const BlockNormGradArgs a) {
    using L = RowLayout<DT, ALIGNED, NV>;
    using E = Elem<DT>;
    using type = typename L::type;
    constexpr int H = L::N / 2, S = kNormGradStages;  // pairs of elements a thread
    extern __shared__ uint4 ring[];
    __shared__ float slots[RowReducer::SLOTS];
    RowReducer red{slots, (int)(blockDim.x >> 5), a.ranks};
    const int threads = blockDim.x, tx = threadIdx.x;
    const int rank = (int)(blockIdx.x % (unsigned)a.ranks), group_id = (int)(blockIdx.x / (unsigned)a.ranks);
    const int c0 = rank * a.width, D = min(a.width, a.D - c0);  // this block's columns
    const float inv_d = 1.f / (float)a.D;
    const int runner = group_id * blockDim.y + threadIdx.y;
    if (runner >= a.runners) return;  // only where a warp is a runner: no barrier spans warps
    const RowRuns runs(a.T, a.runners);
    const int begin = runs.first(runner), end = runs.first(runner + 1);
    const bool token_gate = a.gate_period == 1;
    const int pieces = row_pieces(a.width, sizeof(type));
    const int g_at = 3 * pieces, dr_at = (token_gate ? 4 : 3) * pieces;
    const int stride = dr_at + (a.dr ? pieces : 0);
    uint4 *mine = ring + threadIdx.y * S * stride;

    // registers hold the row, the sums and w_post; w_pre is read again for each row (from L1)
    F2 w_pre[H], w_post[H], dw_pre[H], dw_post[H], dgate[H];
    if (a.w_post) {
        L::weights(a.w_post, a.w_f32, c0, D, threads, tx, w_post);
    } else {
#pragma unroll
        for (int i = 0; i < H; ++i) w_post[i] = F2(1.f);
    }
#pragma unroll
    for (int i = 0; i < H; ++i) dw_pre[i] = dw_post[i] = dgate[i] = F2(0.f);
    float *partial = a.partial + (int64_t)runner * 4 * a.D + c0;  // four sums of a.D columns

    auto put = [&](float *to, const F2 *v) {
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const float2 f = v[i].both();
            const int c = L::col(2 * i, threads, tx), c1 = L::col(2 * i + 1, threads, tx);
            if (c < D) to[c] = f.x;
            if (c1 < D) to[c1] = f.y;
        }
    };

    auto x_row = [&](int64_t t) { return static_cast<const type *>(a.x) + t * a.ldx + c0; };
    auto y_row = [&](int64_t t) { return static_cast<const type *>(a.y) + t * a.ldy + c0; };
    auto n_row = [&](int64_t t) { return static_cast<const type *>(a.dn) + t * a.lddn + c0; };
    auto r_row = [&](int64_t t) { return static_cast<const type *>(a.dr) + t * a.lddr + c0; };
    auto g_row = [&](int64_t g) { return static_cast<const type *>(a.gate) + g * a.ldg + c0; };
    auto fetch = [&](int64_t t, int stage) {
        if (t < end) {
            uint4 *slot = mine + stage * stride;
            L::copy(slot, x_row(t), D, threads, tx);
            L::copy(slot + pieces, y_row(t), D, threads, tx);
            L::copy(slot + 2 * pieces, n_row(t), D, threads, tx);
            if (token_gate) L::copy(slot + g_at, g_row(t), D, threads, tx);
            if (a.dr) L::copy(slot + dr_at, r_row(t), D, threads, tx);
        }
        cp_async_commit();
    };
#pragma unroll
    for (int s = 0; s < S - 1; ++s) fetch(begin + s, s);

    // the gate row of row t, the rows of it behind the runner's first, and the rows left of it
    const int first_group = a.gate_period ? begin / a.gate_period : 0;
    int group = first_group, left = a.gate_period ? a.gate_period - (begin - first_group * a.gate_period) : 0;
    int stage = 0;
    for (int64_t t = begin; t < end; ++t) {
        cp_async_wait<S - 2>();
        if (!ALIGNED) row_sync(red.warps);
        const uint4 *slot = mine + stage * stride;
        fetch(t + S - 1, stage == 0 ? S - 1 : stage - 1);
        stage = stage == S - 1 ? 0 : stage + 1;
        const float rho = a.w_post ? a.rstd[t] : 1.f, rho2 = a.rstd[a.T + t];
        F2 r[H], h[H], u[H], g[H];
        L::read(slot, x_row(t), D, threads, tx, r);
        L::read(slot + pieces, y_row(t), D, threads, tx, h);
        L::read(slot + 2 * pieces, n_row(t), D, threads, tx, u);
        // the factor of dx in the gradient of h
        {
            if (token_gate) {
                L::read(slot + g_at, g_row(t), D, threads, tx, g);
            } else if (a.gate_period) {
                const type *row = g_row(group);  // the same for many rows: from L1
                float v[L::N];
                if constexpr (ALIGNED) {
#pragma unroll
                    for (int k = 0; k < NV; ++k) {
                        const int c = (k * threads + tx) * L::VEC;
                        unpack16<DT>(c < D ? __ldg(reinterpret_cast<const uint4 *>(row + c)) : make_uint4(0, 0, 0, 0),
                                     v + k * L::VEC);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < L::N; ++i) v[i] = i * threads + tx < D ? E::to_float(row[i * threads + tx]) : 0.f;
                }
#pragma unroll
                for (int i = 0; i < H; ++i) g[i] = F2(v[2 * i], v[2 * i + 1]);
            }
#pragma unroll
            for (int i = 0; i < H; ++i) g[i] = a.gate_period ? g[i] * F2(a.scale) : F2(a.scale);
        }
        L::weights(a.w_pre, a.w_f32, c0, D, threads, tx, w_pre);
        F2 part[3] = {F2(0.f), F2(0.f), F2(0.f)}, dr[H];
        if (a.dr) {
            L::read(slot + dr_at, r_row(t), D, threads, tx, dr);
        } else {
#pragma unroll
            for (int i = 0; i < H; ++i) dr[i] = F2(0.f);
        }
#pragma unroll
        for (int i = 0; i < H; ++i) {
            // h becomes y rho; r the residual sum; u = dn w_pre
            h[i] = h[i] * F2(rho);
            const F2 P = g[i] * (h[i] * w_post[i]);
            r[i] = r[i] + P;
            dw_pre[i] = fma(u[i], r[i] * F2(rho2), dw_pre[i]);
            u[i] = u[i] * w_pre[i];
            part[0] = fma(u[i], r[i], part[0]);
            part[1] = fma(P, fma(u[i], F2(rho2), dr[i]), part[1]);
            part[2] = fma(P, r[i], part[2]);
        }
        float sums[3] = {part[0].sum(), part[1].sum(), part[2].sum()};
        red.sum(sums);
        const float c = sums[0] * inv_d * rho2 * rho2;
        // with h = y rho: dy = rho (v - h mean(v h)); without the norm rho is 1 and dy = v
        const float c2 = a.w_post ? fmaf(-rho2 * c, sums[2], sums[1]) * inv_d : 0.f;
#pragma unroll
        for (int i = 0; i < H; ++i) {
            r[i] = fma(fma(r[i], F2(-c), u[i]), F2(rho2), dr[i]);
            dgate[i] = fma(r[i], h[i] * w_post[i], dgate[i]);  // times a.scale when it is written
            u[i] = g[i] * r[i];
            dw_post[i] = fma(u[i], h[i], dw_post[i]);
            u[i] = fma(h[i], F2(-c2), u[i] * w_post[i]) * F2(rho);
        }
        L::store(static_cast<type *>(a.dx) + t * a.lddx + c0, D, threads, tx, r);
        L::store(static_cast<type *>(a.dy) + t * a.lddy + c0, D, threads, tx, u);
        if (a.gate_period && (--left == 0 || t + 1 == end)) {
            // the gate row's sum: whole when all of its rows are this runner's, otherwise one
            // of the runner's two partial sums (the first gate row it meets, or the last)
#pragma unroll
            for (int i = 0; i < H; ++i) dgate[i] = dgate[i] * F2(a.scale);
            if (left == 0 && (group > first_group || begin == group * a.gate_period)) {
                L::store(static_cast<type *>(a.dgate) + group * a.lddg + c0, D, threads, tx, dgate);
            } else {
                put(partial + (int64_t)(group == first_group ? 2 : 3) * a.D, dgate);
            }
            ++group;
            left = a.gate_period;
#pragma unroll
            for (int i = 0; i < H; ++i) dgate[i] = F2(0.f);
        }
    }
    put(partial, dw_pre);
    put(partial + a.D, dw_post);
    if (a.ranks > 1) cluster_sync();
}

// Adds the runners' partial sums: blockIdx.y 0 and 1 for the weights, from 2
// on for the gate rows that more than one runner has a part of.  32 columns by
// 32 slices of the runners, added in slice order.
template <int DT>
__global__ void __launch_bounds__(1024) block_norm_grad_join_kernel(const BlockNormGradArgs a) {
    __shared__ float part[32][33];
    const int D = a.D, c = blockIdx.x * 32 + threadIdx.x, runners = a.runners;
    // the sum over runners [b0, b1) of the partial sum that slot(b) names; valid in slice 0
    auto join = [&](int b0, int b1, auto slot) {
        float s = 0.f;
        if (c < D)
            for (int b = b0 + (int)threadIdx.y; b < b1; b += 32) s += a.partial[((int64_t)b * 4 + slot(b)) * D + c];
        part[threadIdx.y][threadIdx.x] = s;
        __syncthreads();
        if (threadIdx.y == 0)
#pragma unroll
            for (int i = 1; i < 32; ++i) s += part[i][threadIdx.x];
        __syncthreads();
        return s;
    };
    griddep_wait();
    const bool writes = threadIdx.y == 0 && c < D;
    if (blockIdx.y < 2) {
        if (blockIdx.y == 1 && !a.w_post) return;
        const float s = join(0, runners, [&](int) { return (int)blockIdx.y; });
        if (writes) store_weight<DT>(blockIdx.y ? a.dw_post : a.dw_pre, a.w_f32, c, s);
        return;
    }
    // gate rows by number where they are few; otherwise by the runners that start inside one
    const RowRuns runs(a.T, runners);
    const int groups = a.T / a.gate_period, count = min(groups, runners - 1);
    for (int i = blockIdx.y - 2; i < count; i += gridDim.y - 2) {
        int group = i;
        if (groups > runners - 1) {
            const int row = runs.first(i + 1);
            group = row / a.gate_period;
            const int g0 = group * a.gate_period;
            if (g0 == row || runs.first(i) > g0) continue;  // not the first runner to start inside it
        }
        const int g0 = group * a.gate_period;
        const int b0 = runs.runner_of(g0), b1 = runs.runner_of(g0 + a.gate_period - 1) + 1;
        if (b1 - b0 < 2) continue;  // one runner had all of it
        // a runner that starts in an earlier gate row has this one's part in its second place
        const float s = join(b0, b1, [&](int b) { return runs.first(b) >= g0 ? 2 : 3; });
        if (writes) store_weight<DT>(a.dgate, 0, (int64_t)group * a.lddg + c, s);
    }
}

}  // namespace sgemm
