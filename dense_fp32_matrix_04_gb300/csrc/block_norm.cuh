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
// it will read itself and needs no barrier, and its pieces past the row's end
// are zeros that no copy touches, so that what it reads needs no test (a test
// a piece had made half of the gradient's instructions branches and their
// bookkeeping); any other row is copied as the
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
    // zeros past the end of `rows` slots of `pieces` each
    __device__ static void clear(uint4 *slot, int rows, int pieces, int D, int threads, int tx) {
        if (!ALIGNED || D == N * threads) return;
        for (int k = 0; k < rows; ++k)
            for (int p = tx; p < NV * threads; p += threads)
                if (p * VEC >= D) slot[k * pieces + p] = make_uint4(0, 0, 0, 0);
    }
    // this thread's elements of the row that was copied from `row`; 0 past its end
    __device__ static void read(const uint4 *slot, const type *row, int D, int threads, int tx, float *out) {
        if constexpr (ALIGNED) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                unpack16<DT>(slot[v * threads + tx], out + v * VEC);
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
                const int at = (v * threads + tx) * VEC, c = at < D ? at : 0;
                if (w_f32) {
#pragma unroll
                    for (int e = 0; e < VEC; e += 4) {
                        const float4 q = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(w) + c0 + c + e));
                        out[v * VEC + e] = q.x, out[v * VEC + e + 1] = q.y;
                        out[v * VEC + e + 2] = q.z, out[v * VEC + e + 3] = q.w;
                    }
                } else {
                    unpack16<DT>(__ldg(reinterpret_cast<const uint4 *>(static_cast<const type *>(w) + c0 + c)), out + v * VEC);
                }
#pragma unroll
                for (int e = 0; e < VEC; ++e) out[v * VEC + e] = at < D ? out[v * VEC + e] : 0.f;
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                out[i] = i * threads + tx < D ? load_weight<DT>(w, w_f32, c0 + i * threads + tx) : 0.f;
        }
    }
};

// Four elements at a time of an ALIGNED thread's row (its elements 4 q to 4 q + 3), where the
// registers hold no more than that of several rows beside each other; a whole piece of any other.
template <int DT, bool ALIGNED>
struct RowPart {
    using One = RowLayout<DT, ALIGNED, 1>;
    using type = typename One::type;
    static constexpr int VEC = One::VEC, N = ALIGNED ? 4 : VEC, PER = VEC / N;
    __device__ static void unpack(const type *p, F2 (&out)[N / 2]) {
        if constexpr (DT == SGEMM_F32) {
            const float4 f = *reinterpret_cast<const float4 *>(p);
            out[0] = F2(f.x, f.y), out[1] = F2(f.z, f.w);
        } else {
            const uint2 w = *reinterpret_cast<const uint2 *>(p);
            float f[8];
            unpack16<DT>(make_uint4(w.x, w.y, 0, 0), f);
            out[0] = F2(f[0], f[1]), out[1] = F2(f[2], f[3]);
        }
    }
    __device__ static int col(int q, int threads, int tx) { return (q / PER * threads + tx) * VEC + q % PER * N; }
    __device__ static void read(const uint4 *slot, const type *row, int D, int threads, int tx, int q, F2 (&out)[N / 2]) {
        if constexpr (ALIGNED) {
            unpack(reinterpret_cast<const type *>(slot) + col(q, threads, tx), out);
        } else {
            One::read(slot, row, D, threads, q * N * threads + tx, out);
        }
    }
    __device__ static void weights(const void *w, int w_f32, int c0, int D, int threads, int tx, int q, F2 (&out)[N / 2]) {
        if constexpr (ALIGNED) {
            const int at = col(q, threads, tx), c = at < D ? at : 0;
            if (w_f32) {
                const float4 f = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(w) + c0 + c));
                out[0] = F2(f.x, f.y), out[1] = F2(f.z, f.w);
            } else {
                unpack(static_cast<const type *>(w) + c0 + c, out);
            }
            if (at >= D) out[0] = out[1] = F2(0.f);
        } else {
            One::weights(w, w_f32, c0, D, threads, q * N * threads + tx, out);
        }
    }
};

// Rows a thread keeps on their way (and the one it works on).
constexpr int kNormStages = 4;
constexpr int kNormGradStages = 3;

// 16-byte pieces of the slot of one input of a row, for `threads` threads of `per` elements each
// (the last piece for a row that does not start on one).
__host__ __device__ constexpr int row_pieces(int threads, int per, int size) { return threads * per * size / 16 + 1; }

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
    const int arrays = token_gate ? 3 : 2, pieces = row_pieces(threads, N, sizeof(type));
    uint4 *mine = ring + threadIdx.y * S * arrays * pieces;
    L::clear(mine, S * arrays, pieces, D, threads, tx);

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
        L::read(slot, x_row(t), D, threads, tx, r);
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

// The gradient of a row needs, with u = rho2 dn w_pre, m = a g w_post, v = m dx,
//     w = dr + u,   dx = w - r rho2^2 mean(u r),
//     dy = rho v - y rho^3 mean(v y),
// with rho and rho2 from the forward pass.  The second mean need not wait for
// the first:
//     sum(v y) = sum(m y w) - rho2^2 mean(u r) sum(m y r),
// so three sums are taken at once, and a row costs one barrier.
//
// Sums over rows stay in registers: dw_pre, and s = sum(rho y dx), which while
// the gate row is the same is all that the other two need: dgate = a w_post s
// and dw_post += a g s when it changes.  With TOKEN each row has its own gate,
// the sum is dw_post's, and dgate is written with the row.  What a runner has
// of a sum goes to `partial`, where a second kernel adds the runners in order.
template <int DT, bool ALIGNED, int NV, bool TOKEN, int MAXT>
__global__ void __launch_bounds__(MAXT, 1) block_norm_grad_kernel(const BlockNormGradArgs a) {
    using L = RowLayout<DT, ALIGNED, NV>;
    using E = Elem<DT>;
    using type = typename L::type;
    using One = RowLayout<DT, ALIGNED, 1>;  // a piece of a thread's row
    using Part = RowPart<DT, ALIGNED>;
    constexpr int H = L::N / 2, P = One::N / 2, Q = Part::N / 2, S = kNormGradStages;  // pairs of elements
    extern __shared__ uint4 ring[];
    __shared__ float slots[RowReducer::SLOTS];
    RowReducer red{slots, (int)(blockDim.x >> 5), a.ranks};
    const int threads = blockDim.x, tx = threadIdx.x;
    auto first = [&](int v) { return tx + v * (ALIGNED ? 1 : One::N) * threads; };  // as One sees piece v
    const int rank = (int)(blockIdx.x % (unsigned)a.ranks), group_id = (int)(blockIdx.x / (unsigned)a.ranks);
    const int c0 = rank * a.width, D = min(a.width, a.D - c0);  // this block's columns
    const float inv_d = 1.f / (float)a.D;
    const int runner = group_id * blockDim.y + threadIdx.y;
    if (runner >= a.runners) return;  // only where a warp is a runner: no barrier spans warps
    const RowRuns runs(a.T, a.runners);
    const int begin = runs.first(runner), end = runs.first(runner + 1);
    const int pieces = row_pieces(threads, L::N, sizeof(type));
    const int dr_at = (TOKEN ? 4 : 3) * pieces;
    const int stride = dr_at + (a.dr ? pieces : 0);
    uint4 *mine = ring + threadIdx.y * S * stride;
    L::clear(mine, S * stride / pieces, pieces, D, threads, tx);
    // the runner's four sums of a.D columns
    auto partial = [&](int k) { return a.partial + (((int64_t)runner * 4 + k) * a.D + c0); };

    // gate: m above, but w_post alone with TOKEN; s: dw_post with TOKEN
    F2 m[H], dw_pre[H], s[H];
    auto post = [&](int v, F2 *out) {
        if (a.w_post) {
            One::weights(a.w_post, a.w_f32, c0, D, threads, first(v), out);
        } else {
#pragma unroll
            for (int i = 0; i < P; ++i) out[i] = F2(1.f);
        }
    };
    // a g for a gate row: read from L1 where it is the same for many rows
    auto gate_row = [&](int group, int v, F2 *out) {
        if (a.gate_period) {
            One::weights(static_cast<const type *>(a.gate) + group * a.ldg, 0, c0, D, threads, first(v), out);
#pragma unroll
            for (int i = 0; i < P; ++i) out[i] = out[i] * F2(a.scale);
        } else {
#pragma unroll
            for (int i = 0; i < P; ++i) out[i] = F2(a.scale);
        }
    };
    auto take_gate = [&](int group) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            F2 g[P];
            post(v, m + v * P);
            if (TOKEN) continue;
            gate_row(group, v, g);
#pragma unroll
            for (int i = 0; i < P; ++i) m[v * P + i] = m[v * P + i] * g[i];
        }
    };
    // four columns to a store where a thread has four beside each other (single floats would write
    // every sector eight times)
    auto put = [&](float *to, int v, const F2 *q, bool add) {
        if constexpr (ALIGNED) {
            const int c = One::col(0, threads, first(v));
            if (c < D)
#pragma unroll
                for (int i = 0; i < P; i += 2) {
                    float4 *p = reinterpret_cast<float4 *>(to + c + 2 * i);
                    const float2 f = q[i].both(), g = q[i + 1].both();
                    float4 s = make_float4(f.x, f.y, g.x, g.y);
                    if (add) {
                        const float4 o = *p;
                        s = make_float4(o.x + s.x, o.y + s.y, o.z + s.z, o.w + s.w);
                    }
                    *p = s;
                }
        } else {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const float2 f = q[i].both();
                const int c = One::col(2 * i, threads, first(v)), c1 = One::col(2 * i + 1, threads, first(v));
                if (c < D) to[c] = add ? to[c] + f.x : f.x;
                if (c1 < D) to[c1] = add ? to[c1] + f.y : f.y;
            }
        }
    };

    // row t: leading dimensions are 32-bit, so this is one multiplication, and no register holds it
    auto at = [&](const void *p, int64_t ld, int t) { return static_cast<const type *>(p) + ((int64_t)t * (int)ld + c0); };
    auto to = [&](void *p, int64_t ld, int t) { return static_cast<type *>(p) + ((int64_t)t * (int)ld + c0); };
    auto fetch = [&](int t, int stage) {
        if (t < end) {
            uint4 *slot = mine + stage * stride;
            L::copy(slot, at(a.x, a.ldx, t), D, threads, tx);
            L::copy(slot + pieces, at(a.y, a.ldy, t), D, threads, tx);
            L::copy(slot + 2 * pieces, at(a.dn, a.lddn, t), D, threads, tx);
            if (TOKEN) L::copy(slot + 3 * pieces, at(a.gate, a.ldg, t), D, threads, tx);
            if (a.dr) L::copy(slot + dr_at, at(a.dr, a.lddr, t), D, threads, tx);
        }
        cp_async_commit();
    };
#pragma unroll
    for (int k = 0; k < S - 1; ++k) fetch(begin + k, k);

    // the row before which row t's gate row ends
    int last = end;
    if (!TOKEN && a.gate_period) last = (begin / a.gate_period + 1) * a.gate_period;
    take_gate(!TOKEN && a.gate_period ? begin / a.gate_period : 0);
#pragma unroll
    for (int i = 0; i < H; ++i) dw_pre[i] = s[i] = F2(0.f);

    int stage = 0;
    for (int t = begin; t < end; ++t) {
        cp_async_wait<S - 2>();
        if (!ALIGNED) row_sync(red.warps);
        const uint4 *slot = mine + stage * stride;
        fetch(t + S - 1, stage == 0 ? S - 1 : stage - 1);
        stage = stage == S - 1 ? 0 : stage + 1;
        const float rho = a.w_post ? a.rstd[t] : 1.f, rho2 = a.rstd[a.T + t];
        // What the second half needs again is kept (or, y and the gate, read again): a piece at a time
        // the rest fits registers.
        F2 r[H], w[H], part[3] = {F2(0.f), F2(0.f), F2(0.f)};
        auto read_y = [&](int v, F2 *out) {
            One::read(slot + pieces, ALIGNED ? nullptr : at(a.y, a.ldy, t), D, threads, first(v), out);
        };
        auto read_gate = [&](int v, F2 *out) {
            One::read(slot + 3 * pieces, ALIGNED ? nullptr : at(a.gate, a.ldg, t), D, threads, first(v), out);
#pragma unroll
            for (int i = 0; i < P; ++i) out[i] = out[i] * F2(a.scale);
        };
#pragma unroll
        for (int q = 0; q < H / Q; ++q) {
            F2 xx[Q], yy[Q], u[Q], d[Q], w_pre[Q], g[Q];
            Part::read(slot, ALIGNED ? nullptr : at(a.x, a.ldx, t), D, threads, tx, q, xx);
            Part::read(slot + pieces, ALIGNED ? nullptr : at(a.y, a.ldy, t), D, threads, tx, q, yy);
            if constexpr (TOKEN) {
                Part::read(slot + 3 * pieces, ALIGNED ? nullptr : at(a.gate, a.ldg, t), D, threads, tx, q, g);
#pragma unroll
                for (int i = 0; i < Q; ++i) g[i] = g[i] * F2(a.scale);
            }
            Part::read(slot + 2 * pieces, ALIGNED ? nullptr : at(a.dn, a.lddn, t), D, threads, tx, q, u);
            if (a.dr) {
                Part::read(slot + dr_at, ALIGNED ? nullptr : at(a.dr, a.lddr, t), D, threads, tx, q, d);
            } else {
#pragma unroll
                for (int i = 0; i < Q; ++i) d[i] = F2(0.f);
            }
            Part::weights(a.w_pre, a.w_f32, c0, D, threads, tx, q, w_pre);  // again for each row, from L1
#pragma unroll
            for (int i = 0; i < Q; ++i) {
                const int e = q * Q + i;
                F2 my = yy[i] * m[e];
                if constexpr (TOKEN) my = my * g[i];
                r[e] = fma(my, F2(rho), xx[i]);
                u[i] = u[i] * F2(rho2);
                dw_pre[e] = fma(u[i], r[e], dw_pre[e]);
                u[i] = u[i] * w_pre[i];
                w[e] = d[i] + u[i];
                part[0] = fma(u[i], r[e], part[0]);
                part[1] = fma(my, w[e], part[1]);
                part[2] = fma(my, r[e], part[2]);
            }
        }
        float sums[3] = {part[0].sum(), part[1].sum(), part[2].sum()};
        red.sum(sums);
        const float c = sums[0] * inv_d * rho2 * rho2;
        // without the norm of y, rho is 1 and dy is v
        const float k = a.w_post ? fmaf(-c, sums[2], sums[1]) * inv_d * rho * rho * rho : 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            F2 yy[P], g[P];
            read_y(v, yy);
            if constexpr (TOKEN) read_gate(v, g);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int e = v * P + i;
                r[e] = fma(r[e], F2(-c), w[e]);
                F2 d = r[e] * F2(rho);
                if constexpr (TOKEN) {
                    const F2 dy = d * yy[i];
                    s[e] = fma(dy, g[i], s[e]);
                    d = d * (m[e] * g[i]);
                    g[i] = dy * m[e] * F2(a.scale);
                } else {
                    s[e] = fma(d, yy[i], s[e]);
                    d = d * m[e];
                }
                w[e] = fma(yy[i], F2(-k), d);
            }
            One::store(to(a.dx, a.lddx, t), D, threads, first(v), r + v * P);
            One::store(to(a.dy, a.lddy, t), D, threads, first(v), w + v * P);
            if constexpr (TOKEN) One::store(to(a.dgate, a.lddg, t), D, threads, first(v), g);
        }
        if (!TOKEN && (t + 1 == last || t + 1 == end)) {
            // a gate row's sum is whole when all of its rows are this runner's, otherwise one of the
            // runner's two partial sums (the first gate row it meets, or the last)
            const bool later = last - a.gate_period > begin;
            const bool whole = t + 1 == last && begin <= last - a.gate_period;
            const int group = a.gate_period ? t / a.gate_period : 0;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                F2 q[P];
                if (a.w_post) {
                    gate_row(group, v, q);
#pragma unroll
                    for (int i = 0; i < P; ++i) q[i] = q[i] * s[v * P + i];
                    put(partial(1), v, q, a.gate_period && later);
                }
                if (a.gate_period) {
                    post(v, q);
#pragma unroll
                    for (int i = 0; i < P; ++i) q[i] = q[i] * s[v * P + i] * F2(a.scale);
                    if (whole) One::store(to(a.dgate, a.lddg, group), D, threads, first(v), q);
                    else put(partial(later ? 3 : 2), v, q, false);
                }
#pragma unroll
                for (int i = 0; i < P; ++i) s[v * P + i] = F2(0.f);
            }
            last += a.gate_period;
            if (t + 1 < end) take_gate(group + 1);
        }
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        put(partial(0), v, dw_pre + v * P, false);
        if (TOKEN) put(partial(1), v, s + v * P, false);
    }
    if (a.ranks > 1) cluster_sync();
}

// Adds the runners' partial sums: blockIdx.y 0 and 1 for the weights, from 2
// on for the gate rows that more than one runner has a part of.  32 columns by
// kNormJoinSlices slices of the runners, each added in order with LOADS loads on
// their way, then the slices in order.
constexpr int kNormJoinSlices = 16;
template <int DT>
__global__ void __launch_bounds__(32 * kNormJoinSlices) block_norm_grad_join_kernel(const BlockNormGradArgs a) {
    constexpr int LOADS = 16;
    __shared__ float part[kNormJoinSlices][32];
    const int D = a.D, c = blockIdx.x * 32 + threadIdx.x, runners = a.runners;
    // the sum over runners [b0, b1) of their partial sum k, or k3 for those below b3 <= b0 + 1;
    // valid in slice 0
    auto join = [&](int b0, int b1, int k, int k3, int b3) {
        float s = 0.f;
        const int64_t step = (int64_t)kNormJoinSlices * 4 * D;
        if (c < D) {
            int b = b0 + (int)threadIdx.y;
            if (b < b3) {
                s = a.partial[((int64_t)b * 4 + k3) * D + c];
                b += kNormJoinSlices;
            }
            const float *p = a.partial + ((int64_t)b * 4 + k) * D + c;
            for (; b < b1; b += LOADS * kNormJoinSlices, p += LOADS * step) {
                float v[LOADS];
#pragma unroll
                for (int i = 0; i < LOADS; ++i) v[i] = b + i * kNormJoinSlices < b1 ? __ldcg(p + i * step) : 0.f;
#pragma unroll
                for (int i = 0; i < LOADS; ++i) s += v[i];
            }
        }
        part[threadIdx.y][threadIdx.x] = s;
        __syncthreads();
        if (threadIdx.y == 0)
#pragma unroll
            for (int i = 1; i < kNormJoinSlices; ++i) s += part[i][threadIdx.x];
        __syncthreads();
        return s;
    };
    griddep_wait();
    const bool writes = threadIdx.y == 0 && c < D;
    if (blockIdx.y < 2) {
        if (blockIdx.y == 1 && !a.w_post) return;
        const float s = join(0, runners, (int)blockIdx.y, 0, 0);
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
        // a runner that starts in an earlier gate row (the first one here) has this one's part in its
        // second place
        const float s = join(b0, b1, 2, 3, runs.first(b0) < g0 ? b0 + 1 : b0);
        if (writes) store_weight<DT>(a.dgate, 0, (int64_t)group * a.lddg + c, s);
    }
}

}  // namespace sgemm
