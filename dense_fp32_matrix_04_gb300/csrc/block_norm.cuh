// The norms, gate and residual sum between two blocks of a model, and their
// gradient:
//     h = y rho w_post,  rho = rsqrt(mean(y^2) + eps)
//     r = x + a g h
//     n = r rho2 w_pre,  rho2 = rsqrt(mean(r^2) + eps)
// A row is read once into registers, its two sums of squares are reduced over
// the threads that share it, and r and n are written once.
//
// Memory bounds the forward pass: four elements moved for about ten operations.
// 8192 x 5120 BF16 takes 58.6 us, 5.7 TB/s of the 6.8 that a copy reaches; a
// row's two barriers are what is left.  Rows are walked by blocks that stay, so
// that copies of the next three rows are always on their way (a test and an
// address for each piece took 63 us).  Seven rows of 4096 take 3.8 us, a launch
// and two memory latencies.
//
// The gradient moves six elements for about 25 operations: 8192 x 4096 BF16
// takes 84 us (4.8 TB/s), FP32 4096 x 4096, half the arithmetic for the same
// bytes, 79; 9 us of it are the launch, the runners' first row and the joining
// of their sums.  Rows of single elements (not 16-byte aligned, or of odd width)
// run at half of that and less: 2047 x 1111 FP32 takes 24.6 us, the forward pass of
// 8192 x 1111 BF16 37.6 (1112 columns 21.4), of 8192 x 5121 133 (5120 58.6).
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
// flight does not depend on how many blocks fit an SM.
//
// With ALIGNED rows (16-byte aligned and a whole number of pieces) a warp takes
// NV pieces a lane beside each other, so that one address serves all of them.
// Each thread copies the pieces it will read itself and needs no barrier; its
// pieces past the row's end are copies of nothing, zeros, so that what it reads
// needs no test.  (With a test a piece, and with addresses of their own,
// two thirds of the gradient's instructions were addresses and branches.)
//
// Any other row is copied as the pieces that enclose it (up to 15 bytes in
// front and behind are read and never used), a barrier lets the row's threads
// see each other's copies, and they read single elements, i-th at column
// i * threads + thread.
// 16-byte pieces of the slot of one input of a row, for `threads` threads of `per` elements each
// (the last piece for a row that does not start on one).
__host__ __device__ constexpr int row_pieces(int threads, int per, int size) { return threads * per * size / 16 + 1; }

template <int DT, bool ALIGNED, int NV>
struct RowLayout {
    using type = typename Elem<DT>::type;
    static constexpr int VEC = Elem<DT>::VEC, N = NV * VEC;  // elements a thread
    static constexpr int NEXT = 32 * VEC;                    // columns from a thread's piece to its next
    int D, threads, tx;
    int col, left;  // ALIGNED: this thread's first column, and the columns from there to the row's end

    __device__ explicit RowLayout(int D) : D(D), threads(blockDim.x), tx(threadIdx.x) {
        col = ALIGNED ? ((tx & ~31) * NV + (tx & 31)) * VEC : 0;
        left = D - col;
    }
    // pieces of the slot of one input, and a thread's place in the ring of `rows` slots
    __device__ int pieces() const { return ALIGNED ? NV * 32 : row_pieces(threads, N, sizeof(type)); }
    __device__ uint4 *place(uint4 *ring, int rows) const {
        if constexpr (ALIGNED) {
            const int warp = (threadIdx.y * threads + tx) >> 5;
            return ring + warp * rows * pieces() + (tx & 31);
        } else {
            return ring + threadIdx.y * rows * pieces();
        }
    }
    __device__ bool has(int e) const { return left > e / VEC * NEXT; }  // ALIGNED: the piece of element e
    __device__ static int at(int e) { return e / VEC * NEXT + e % VEC; }
    // The functions below take rows from this thread's first column (ALIGNED) or their start, and
    // slots from this thread's place.
    __device__ void copy(uint4 *slot, const type *row) const {
        if constexpr (ALIGNED) {
#pragma unroll
            for (int v = 0; v < NV; ++v)
                cp_async_16(smem_addr(slot + v * 32), row + v * NEXT, has(v * VEC) ? 16 : 0);
        } else {
            const uintptr_t lo = reinterpret_cast<uintptr_t>(row) & ~(uintptr_t)15;
            const int n = (int)((reinterpret_cast<uintptr_t>(row + D) + 15 - lo) >> 4);
            for (int p = tx; p < n; p += threads)
                cp_async_16(smem_addr(slot + p), reinterpret_cast<const void *>(lo + 16 * (uintptr_t)p), 16);
        }
    }
    template <int COUNT>
    __device__ static void unpack(const type *p, F2 (&out)[COUNT / 2]) {
        float f[8];
        if constexpr (sizeof(type) * COUNT == 16) {
            unpack16<DT>(*reinterpret_cast<const uint4 *>(p), f);
        } else {
            const uint2 w = *reinterpret_cast<const uint2 *>(p);
            unpack16<DT>(make_uint4(w.x, w.y, 0, 0), f);
        }
#pragma unroll
        for (int i = 0; i < COUNT / 2; ++i) out[i] = F2(f[2 * i], f[2 * i + 1]);
    }
    // COUNT elements (a piece, or four of one) from this thread's e-th of the row that was copied
    // from `row`; 0 past its end
    template <int COUNT>
    __device__ void read(const uint4 *slot, const type *row, int e, F2 (&out)[COUNT / 2]) const {
        if constexpr (ALIGNED) {
            unpack<COUNT>(reinterpret_cast<const type *>(slot + e / VEC * 32) + e % VEC, out);
        } else {
            const type *q = reinterpret_cast<const type *>(slot) + (reinterpret_cast<uintptr_t>(row) & 15) / sizeof(type);
            auto one = [&](int i) { return i * threads + tx < D ? Elem<DT>::to_float(q[i * threads + tx]) : 0.f; };
#pragma unroll
            for (int i = 0; i < COUNT; i += 2) out[i / 2] = F2(one(e + i), one(e + i + 1));
        }
    }
    // the same of weights (from the block's first column); ALIGNED weights start on 16 bytes.
    // FOR_ZEROS: they meet only zeros past the row's end, and are the row's last ones there.
    template <int COUNT, bool FOR_ZEROS = false>
    __device__ void weights(const void *w, int w_f32, int e, F2 (&out)[COUNT / 2]) const {
        if constexpr (ALIGNED && FOR_ZEROS) {
            const int c = (has(e) ? col + e / VEC * NEXT : D - VEC) + e % VEC;
            if (w_f32) {
#pragma unroll
                for (int i = 0; i < COUNT; i += 4) {
                    const float4 f = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(w) + c + i));
                    out[i / 2] = F2(f.x, f.y), out[i / 2 + 1] = F2(f.z, f.w);
                }
            } else {
                unpack<COUNT>(static_cast<const type *>(w) + c, out);
            }
        } else if constexpr (ALIGNED) {
#pragma unroll
            for (int i = 0; i < COUNT / 2; ++i) out[i] = F2(0.f);
            if (w_f32) {
#pragma unroll
                for (int i = 0; i < COUNT; i += 4)
                    if (has(e)) {
                        const float4 f = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(w) + col + at(e + i)));
                        out[i / 2] = F2(f.x, f.y), out[i / 2 + 1] = F2(f.z, f.w);
                    }
            } else if (has(e)) {
                unpack<COUNT>(static_cast<const type *>(w) + col + at(e), out);
            }
        } else {
            auto one = [&](int i) { return i * threads + tx < D ? load_weight<DT>(w, w_f32, i * threads + tx) : 0.f; };
#pragma unroll
            for (int i = 0; i < COUNT; i += 2) out[i / 2] = F2(one(e + i), one(e + i + 1));
        }
    }
    // a piece from this thread's e-th element on
    __device__ void store(type *row, int e, const F2 *v) const {
        float f[VEC];
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
            const float2 b = v[i].both();
            f[2 * i] = b.x;
            f[2 * i + 1] = b.y;
        }
        if constexpr (ALIGNED) {
            if (has(e)) *reinterpret_cast<uint4 *>(row + at(e)) = pack16<DT>(f);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if ((e + i) * threads + tx < D) row[(e + i) * threads + tx] = Elem<DT>::from_float(f[i]);
        }
    }
    // the same of FP32 sums, four columns to a store where a thread has them beside each other
    // (single floats would write every sector eight times)
    __device__ void put(float *row, int e, const F2 *v, bool add) const {
        if constexpr (ALIGNED) {
            if (has(e))
#pragma unroll
                for (int i = 0; i < VEC / 2; i += 2) {
                    float4 *p = reinterpret_cast<float4 *>(row + at(e + 2 * i));
                    const float2 f = v[i].both(), g = v[i + 1].both();
                    float4 s = make_float4(f.x, f.y, g.x, g.y);
                    if (add) {
                        const float4 o = *p;
                        s = make_float4(o.x + s.x, o.y + s.y, o.z + s.z, o.w + s.w);
                    }
                    *p = s;
                }
        } else {
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) {
                const float2 f = v[i].both();
                const int c = (e + 2 * i) * threads + tx, c1 = c + threads;
                if (c < D) row[c] = add ? row[c] + f.x : f.x;
                if (c1 < D) row[c1] = add ? row[c1] + f.y : f.y;
            }
        }
    }
};

// Rows a thread keeps on their way (and the one it works on).
constexpr int kNormStages = 4;
constexpr int kNormGradStages = 3;

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
    constexpr int N = L::N, V = L::VEC, H = V / 2, S = kNormStages;  // H pairs a piece
    extern __shared__ uint4 ring[];
    __shared__ float slots[RowReducer::SLOTS];
    RowReducer red{slots, (int)(blockDim.x >> 5), a.ranks};
    const int rank = (int)(blockIdx.x % (unsigned)a.ranks), group_id = (int)(blockIdx.x / (unsigned)a.ranks);
    const int c0 = rank * a.width;  // this block's columns
    const L l(min(a.width, a.D - c0));
    const int cols = c0 + l.col;
    const float inv_d = 1.f / (float)a.D;
    const bool token_gate = a.gate_period == 1;
    const int arrays = token_gate ? 3 : 2, pieces = l.pieces();
    uint4 *mine = l.place(ring, S * arrays);

    auto weights = [&](const void *w, int v, F2 (&out)[H]) {
        l.template weights<V>(static_cast<const char *>(w) + (int64_t)c0 * (a.w_f32 ? 4 : (int)sizeof(type)), a.w_f32, v * V, out);
    };
    F2 w_pre[NV][H], w_post[NV][H];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        weights(a.w_pre, v, w_pre[v]);
        if (a.w_post) weights(a.w_post, v, w_post[v]);
    }

    const int64_t first = (int64_t)group_id * blockDim.y + threadIdx.y;
    const int64_t step = (int64_t)(gridDim.x / (unsigned)a.ranks) * blockDim.y;
    // rows are numbered below 2^30 and leading dimensions are 32-bit: one multiplication
    auto row = [&](const void *p, int64_t ld, int64_t t) {
        return static_cast<const type *>(p) + ((int64_t)(int)t * (int)ld + cols);
    };
    auto x_row = [&](int64_t t) { return row(a.x, a.ldx, t); };
    auto y_row = [&](int64_t t) { return row(a.y, a.ldy, t); };
    auto g_row = [&](int64_t t) { return row(a.gate, a.ldg, (unsigned)t / (unsigned)a.gate_period); };
    auto fetch = [&](int64_t t, int stage) {
        if (t < a.T) {
            uint4 *slot = mine + stage * arrays * pieces;
            l.copy(slot, x_row(t));
            l.copy(slot + pieces, y_row(t));
            if (token_gate) l.copy(slot + 2 * pieces, g_row(t));
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
        F2 h[NV][H], r[NV][H];
#pragma unroll
        for (int v = 0; v < NV; ++v) l.template read<V>(slot + pieces, y_row(t), v * V, h[v]);
        float rho = 1.f;
        if (a.w_post) {
            F2 ss(0.f);
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int i = 0; i < H; ++i) ss = fma(h[v][i], h[v][i], ss);
            rho = rsqrtf(fmaf(red.sum(ss.sum()), inv_d, a.eps));
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int i = 0; i < H; ++i) h[v][i] = h[v][i] * (F2(rho) * w_post[v][i]);
        }
        if (a.gate_period) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                F2 g[H];
                if (token_gate) l.template read<V>(slot + 2 * pieces, g_row(t), v * V, g);
                else l.template weights<V>(g_row(t) - l.col, 0, v * V, g);  // the same for many rows: from L1
#pragma unroll
                for (int i = 0; i < H; ++i) h[v][i] = h[v][i] * g[i];
            }
        }
        // the slot that the previous row was read from takes the row after the next ones
        fetch(t + (S - 1) * step, stage == 0 ? S - 1 : stage - 1);
        stage = stage == S - 1 ? 0 : stage + 1;
        F2 ss(0.f);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            l.template read<V>(slot, x_row(t), v * V, r[v]);
#pragma unroll
            for (int i = 0; i < H; ++i) {
                r[v][i] = fma(F2(a.scale), h[v][i], r[v][i]);
                ss = fma(r[v][i], r[v][i], ss);
            }
            l.store(const_cast<type *>(row(a.r, a.ldr, t)), v * V, r[v]);
        }
        const float rho2 = rsqrtf(fmaf(red.sum(ss.sum()), inv_d, a.eps));
        if (a.rstd && threadIdx.x == 0 && rank == 0) {
            a.rstd[t] = rho;
            a.rstd[a.T + t] = rho2;
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
#pragma unroll
            for (int i = 0; i < H; ++i) r[v][i] = r[v][i] * (F2(rho2) * w_pre[v][i]);
            if (a.n) l.store(const_cast<type *>(row(a.n, a.ldn, t)), v * V, r[v]);
        }
        if (a.q) {
            uint32_t top = 0;
            float n[N];
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                const float2 f = r[i / V][i % V / 2].both();
                n[i] = f.x;
                n[i + 1] = f.y;
                top = max(top, max(__float_as_uint(f.x) & 0x7fffffffu, __float_as_uint(f.y) & 0x7fffffffu));
            }
            const I8Scale q(red.max(top));
            if (threadIdx.x == 0 && rank == 0) a.q_scale[t] = q.scale;
            int8_t *out = a.q + t * a.ldq + cols;
            if constexpr (ALIGNED) {
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    if (!l.has(v * V)) continue;
                    int8_t b[V];
#pragma unroll
                    for (int e = 0; e < V; ++e) b[e] = q(n[v * V + e]);
                    store_bytes(out + l.at(v * V), b, a.q_vec);
                }
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (i * l.threads + l.tx < l.D) out[i * l.threads + l.tx] = q(n[i]);
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
    using type = typename L::type;
    constexpr int N = L::N, V = L::VEC, P = V / 2, S = kNormGradStages;  // P pairs a piece
    // elements at a time of the first pass, where the registers hold no more of four rows
    constexpr int Q = ALIGNED ? 4 : V;
    extern __shared__ uint4 ring[];
    __shared__ float slots[RowReducer::SLOTS];
    RowReducer red{slots, (int)(blockDim.x >> 5), a.ranks};
    const int rank = (int)(blockIdx.x % (unsigned)a.ranks), group_id = (int)(blockIdx.x / (unsigned)a.ranks);
    const int c0 = rank * a.width;  // this block's columns
    const L l(min(a.width, a.D - c0));
    const int cols = c0 + l.col;
    const float inv_d = 1.f / (float)a.D;
    const int runner = group_id * blockDim.y + threadIdx.y;
    if (runner >= a.runners) return;  // only where a warp is a runner: no barrier spans warps
    const RowRuns runs(a.T, a.runners);
    const int begin = runs.first(runner), end = runs.first(runner + 1);
    constexpr int DR = TOKEN ? 4 : 3;  // slots of a row: x, y, dn, with TOKEN the gate, dr if there is one
    const int pieces = l.pieces(), stride = (a.dr ? DR + 1 : DR) * pieces;
    uint4 *mine = l.place(ring, S * (a.dr ? DR + 1 : DR));
    // the runner's four sums of a.D columns
    auto partial = [&](int k) { return a.partial + (((int64_t)runner * 4 + k) * a.D + cols); };

    // m: as above, but w_post alone with TOKEN; s: dw_post with TOKEN
    F2 m[N / 2], dw_pre[N / 2], s[N / 2];
    const int wsize = a.w_f32 ? 4 : (int)sizeof(type);
    auto post = [&](int v, F2 (&out)[P]) {
        if (a.w_post) {
            l.template weights<V>(static_cast<const char *>(a.w_post) + c0 * wsize, a.w_f32, v * V, out);
        } else {
#pragma unroll
            for (int i = 0; i < P; ++i) out[i] = F2(1.f);
        }
    };
    // a g for a gate row: read from L1 where it is the same for many rows
    auto gate_row = [&](int group, int v, F2 (&out)[P]) {
        if (a.gate_period) {
            l.template weights<V>(static_cast<const type *>(a.gate) + (group * a.ldg + c0), 0, v * V, out);
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
            F2 g[P], w[P];
            post(v, w);
            if (!TOKEN) gate_row(group, v, g);
#pragma unroll
            for (int i = 0; i < P; ++i) m[v * P + i] = TOKEN ? w[i] : w[i] * g[i];
        }
    };

    // row t: leading dimensions are 32-bit, so this is one multiplication, and no register holds it
    auto at = [&](const void *p, int64_t ld, int t) { return static_cast<const type *>(p) + ((int64_t)t * (int)ld + cols); };
    auto to = [&](void *p, int64_t ld, int t) { return static_cast<type *>(p) + ((int64_t)t * (int)ld + cols); };
    auto fetch = [&](int t, int stage) {
        if (t < end) {
            uint4 *slot = mine + stage * stride;
            l.copy(slot, at(a.x, a.ldx, t));
            l.copy(slot + pieces, at(a.y, a.ldy, t));
            l.copy(slot + 2 * pieces, at(a.dn, a.lddn, t));
            if (TOKEN) l.copy(slot + 3 * pieces, at(a.gate, a.ldg, t));
            if (a.dr) l.copy(slot + DR * pieces, at(a.dr, a.lddr, t));
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
    for (int i = 0; i < N / 2; ++i) dw_pre[i] = s[i] = F2(0.f);

    int stage = 0;
    for (int t = begin; t < end; ++t) {
        cp_async_wait<S - 2>();
        if (!ALIGNED) row_sync(red.warps);
        const uint4 *slot = mine + stage * stride;
        fetch(t + S - 1, stage == 0 ? S - 1 : stage - 1);
        stage = stage == S - 1 ? 0 : stage + 1;
        const float rho = a.w_post ? a.rstd[t] : 1.f, rho2 = a.rstd[a.T + t];
        // What the second half needs again is kept (or, y and the gate, read again): a few elements
        // at a time the rest fits registers.
        F2 r[N / 2], w[N / 2], part[3] = {F2(0.f), F2(0.f), F2(0.f)};
#pragma unroll
        for (int e = 0; e < N; e += Q) {
            F2 xx[Q / 2], yy[Q / 2], u[Q / 2], d[Q / 2], w_pre[Q / 2], g[Q / 2];
            l.template read<Q>(slot, at(a.x, a.ldx, t), e, xx);
            l.template read<Q>(slot + pieces, at(a.y, a.ldy, t), e, yy);
            if constexpr (TOKEN) {
                l.template read<Q>(slot + 3 * pieces, at(a.gate, a.ldg, t), e, g);
#pragma unroll
                for (int i = 0; i < Q / 2; ++i) g[i] = g[i] * F2(a.scale);
            }
            l.template read<Q>(slot + 2 * pieces, at(a.dn, a.lddn, t), e, u);
            if (a.dr) {
                l.template read<Q>(slot + DR * pieces, at(a.dr, a.lddr, t), e, d);
            } else {
#pragma unroll
                for (int i = 0; i < Q / 2; ++i) d[i] = F2(0.f);
            }
            // again for each row, from L1
            l.template weights<Q, true>(static_cast<const char *>(a.w_pre) + c0 * wsize, a.w_f32, e, w_pre);
#pragma unroll
            for (int i = 0; i < Q / 2; ++i) {
                const int k = e / 2 + i;
                F2 my = yy[i] * m[k];
                if constexpr (TOKEN) my = my * g[i];
                r[k] = fma(my, F2(rho), xx[i]);
                u[i] = u[i] * F2(rho2);
                dw_pre[k] = fma(u[i], r[k], dw_pre[k]);
                u[i] = u[i] * w_pre[i];
                w[k] = d[i] + u[i];
                part[0] = fma(u[i], r[k], part[0]);
                part[1] = fma(my, w[k], part[1]);
                part[2] = fma(my, r[k], part[2]);
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
            l.template read<V>(slot + pieces, at(a.y, a.ldy, t), v * V, yy);
            if constexpr (TOKEN) l.template read<V>(slot + 3 * pieces, at(a.gate, a.ldg, t), v * V, g);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int e = v * P + i;
                r[e] = fma(r[e], F2(-c), w[e]);
                F2 d = r[e] * F2(rho);
                if constexpr (TOKEN) {
                    g[i] = g[i] * F2(a.scale);
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
            l.store(to(a.dx, a.lddx, t), v * V, r + v * P);
            l.store(to(a.dy, a.lddy, t), v * V, w + v * P);
            if constexpr (TOKEN) l.store(to(a.dgate, a.lddg, t), v * V, g);
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
                    l.put(partial(1), v * V, q, a.gate_period && later);
                }
                if (a.gate_period) {
                    post(v, q);
#pragma unroll
                    for (int i = 0; i < P; ++i) q[i] = q[i] * s[v * P + i] * F2(a.scale);
                    if (whole) l.store(to(a.dgate, a.lddg, group), v * V, q);
                    else l.put(partial(later ? 3 : 2), v * V, q, false);
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
        l.put(partial(0), v * V, dw_pre + v * P, false);
        if (TOKEN) l.put(partial(1), v * V, s + v * P, false);
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
