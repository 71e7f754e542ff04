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
    float *partial;    // blocks x 4 x D: dw_pre, dw_post, and the gate rows a block holds a part of
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

// blockDim.x threads share a row; blockDim.y rows run side by side in a block
// (more than one only where a warp is enough for a row).
// Up to MAXT = 512 threads the weights stay in registers from row to row; 1024
// threads have half the registers and read them again (from L1).
template <int DT, int VW, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT, 1) block_norm_kernel(const BlockNormArgs a) {
    using P = Piece<DT, VW>;
    using type = typename P::type;
    __shared__ float slots[64];
    RowReducer red{slots, (int)(blockDim.x >> 5)};
    const int threads = blockDim.x, D = a.D;
    const float inv_d = 1.f / (float)D;

    constexpr bool KEEP = MAXT <= 512;
    float w_pre[NV * VW], w_post[NV * VW];
    auto load_weights = [&](float *w, const void *from) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int e = 0; e < VW; ++e) {
                const int c = (v * threads + (int)threadIdx.x) * VW + e;
                w[v * VW + e] = c < D ? load_weight<DT>(from, a.w_f32, c) : 0.f;
            }
    };
    if (KEEP) {
        load_weights(w_pre, a.w_pre);
        if (a.w_post) load_weights(w_post, a.w_post);
    }

    const int step = gridDim.x * blockDim.y;
    for (int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; t < a.T; t += step) {
        const type *x = static_cast<const type *>(a.x) + t * a.ldx;
        const type *y = static_cast<const type *>(a.y) + t * a.ldy;
        typename P::raw rx[NV], ry[NV], rg[NV];
        const type *gate =
            a.gate_period ? static_cast<const type *>(a.gate) + (t / a.gate_period) * a.ldg : nullptr;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * threads + (int)threadIdx.x) * VW;
            rx[v] = c < D ? P::load(x + c) : P::zero();
            ry[v] = c < D ? P::load(y + c) : P::zero();
            if (gate) rg[v] = c < D ? P::load(gate + c) : P::zero();
        }
        float h[NV * VW], r[NV * VW];
        float ss = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            P::unpack(ry[v], h + v * VW);
            P::unpack(rx[v], r + v * VW);
        }
        float rho = 1.f;
        if (a.w_post) {
#pragma unroll
            for (int i = 0; i < NV * VW; ++i) ss = fmaf(h[i], h[i], ss);
            rho = rsqrtf(fmaf(red.sum(ss), inv_d, a.eps));
            if (!KEEP) load_weights(w_post, a.w_post);
        }
        ss = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float g[VW];
            if (gate) P::unpack(rg[v], g);
#pragma unroll
            for (int e = 0; e < VW; ++e) {
                const int i = v * VW + e;
                float hv = a.w_post ? h[i] * rho * w_post[i] : h[i];
                if (gate) hv *= g[e];
                r[i] = fmaf(a.scale, hv, r[i]);
                ss = fmaf(r[i], r[i], ss);
            }
        }
        const float rho2 = rsqrtf(fmaf(red.sum(ss), inv_d, a.eps));
        if (a.rstd && threadIdx.x == 0) {
            a.rstd[t] = rho;
            a.rstd[a.T + t] = rho2;
        }
        if (!KEEP) load_weights(w_pre, a.w_pre);
        type *out_r = static_cast<type *>(a.r) + t * a.ldr;
        uint32_t top = 0;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * threads + (int)threadIdx.x) * VW;
            if (c < D) P::store(out_r + c, r + v * VW);
#pragma unroll
            for (int e = 0; e < VW; ++e) {
                const int i = v * VW + e;
                r[i] = r[i] * rho2 * w_pre[i];
                top = max(top, __float_as_uint(r[i]) & 0x7fffffffu);
            }
            if (a.n && c < D) P::store(static_cast<type *>(a.n) + t * a.ldn + c, r + v * VW);
        }
        if (a.q) {
            const I8Scale q(red.max(top));
            if (threadIdx.x == 0) a.q_scale[t] = q.scale;
            int8_t *out = a.q + t * a.ldq;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int c = (v * threads + (int)threadIdx.x) * VW;
                if (c >= D) continue;
                int8_t b[VW];
#pragma unroll
                for (int e = 0; e < VW; ++e) b[e] = q(r[v * VW + e]);
                store_bytes(out + c, b, a.q_vec);
            }
        }
    }
}

// Rows too wide for the registers of a block: one block per row reads it
// again for each step (three times in all; the later reads come from L2).
template <int DT>
__global__ void __launch_bounds__(1024, 1) block_norm_wide_kernel(const BlockNormArgs a) {
    using E = Elem<DT>;
    using type = typename E::type;
    __shared__ float slots[64];
    RowReducer red{slots, (int)(blockDim.x >> 5)};
    const int D = a.D;
    const float inv_d = 1.f / (float)D;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const type *x = static_cast<const type *>(a.x) + t * a.ldx;
        const type *y = static_cast<const type *>(a.y) + t * a.ldy;
        const type *gate =
            a.gate_period ? static_cast<const type *>(a.gate) + (t / a.gate_period) * a.ldg : nullptr;
        float rho = 1.f, ss = 0.f;
        if (a.w_post) {
            for (int c = threadIdx.x; c < D; c += blockDim.x) {
                const float v = E::to_float(y[c]);
                ss = fmaf(v, v, ss);
            }
            rho = rsqrtf(fmaf(red.sum(ss), inv_d, a.eps));
        }
        auto residual = [&](int c) {
            float h = E::to_float(y[c]);
            if (a.w_post) h = h * rho * load_weight<DT>(a.w_post, a.w_f32, c);
            if (gate) h *= E::to_float(gate[c]);
            return fmaf(a.scale, h, E::to_float(x[c]));
        };
        ss = 0.f;
        for (int c = threadIdx.x; c < D; c += blockDim.x) {
            const float r = residual(c);
            ss = fmaf(r, r, ss);
        }
        const float rho2 = rsqrtf(fmaf(red.sum(ss), inv_d, a.eps));
        if (a.rstd && threadIdx.x == 0) {
            a.rstd[t] = rho;
            a.rstd[a.T + t] = rho2;
        }
        I8Scale q(0u);
        if (a.q) {
            uint32_t top = 0;
            for (int c = threadIdx.x; c < D; c += blockDim.x)
                top = max(top, __float_as_uint(residual(c) * rho2 * load_weight<DT>(a.w_pre, a.w_f32, c)) & 0x7fffffffu);
            q = I8Scale(red.max(top));
            if (threadIdx.x == 0) a.q_scale[t] = q.scale;
        }
        // r may be x: each element is read before the same thread writes it
        for (int c = threadIdx.x; c < D; c += blockDim.x) {
            const float r = residual(c);
            const float n = r * rho2 * load_weight<DT>(a.w_pre, a.w_f32, c);
            static_cast<type *>(a.r)[t * a.ldr + c] = E::from_float(r);
            if (a.n) static_cast<type *>(a.n)[t * a.ldn + c] = E::from_float(n);
            if (a.q) a.q[t * a.ldq + c] = q(n);
        }
    }
}

// ---------------------------------------------------------------- gradient

// Block b takes the rows [first_row(b), first_row(b + 1)): consecutive rows,
// so that a gate row's sum stays in registers until the row changes.
__device__ __forceinline__ int block_first_row(int b, int T, int blocks) {
    return (int)((int64_t)b * T / blocks);
}

// The gradient of a row needs, with u = dn w_pre and v = dh w_post,
//     dx = dr + rho2 (u - r rho2^2 mean(u r)),   dh = a g dx,
//     dy = rho (v - y rho^2 mean(v y)),
// so two sums over the row, one after the other; rho and rho2 come from the
// forward pass.  Sums over rows (weights and gate) are kept in registers, and
// written per block to `partial`: a second kernel adds the blocks in order.
template <int DT, int VW, int NV>
__global__ void __launch_bounds__(512, 1) block_norm_grad_kernel(const BlockNormGradArgs a) {
    using P = Piece<DT, VW>;
    using E = Elem<DT>;
    using type = typename P::type;
    constexpr int N = NV * VW;
    __shared__ float slots[64];
    RowReducer red{slots, (int)(blockDim.x >> 5)};
    const int threads = blockDim.x, D = a.D;
    const float inv_d = 1.f / (float)D;
    const int begin = block_first_row(blockIdx.x, a.T, gridDim.x);
    const int end = block_first_row(blockIdx.x + 1, a.T, gridDim.x);

    float w_pre[N], w_post[N], dw_pre[N], dw_post[N], dgate[N];
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < VW; ++e) {
            const int c = (v * threads + (int)threadIdx.x) * VW + e;
            const int i = v * VW + e;
            w_pre[i] = c < D ? load_weight<DT>(a.w_pre, a.w_f32, c) : 0.f;
            w_post[i] = c < D && a.w_post ? load_weight<DT>(a.w_post, a.w_f32, c) : 1.f;
            dw_pre[i] = dw_post[i] = dgate[i] = 0.f;
        }
    float *partial = a.partial + (int64_t)blockIdx.x * 4 * D;

    for (int64_t t = begin; t < end; ++t) {
        const type *x = static_cast<const type *>(a.x) + t * a.ldx;
        const type *y = static_cast<const type *>(a.y) + t * a.ldy;
        const type *pn = static_cast<const type *>(a.dn) + t * a.lddn;
        const type *pr = a.dr ? static_cast<const type *>(a.dr) + t * a.lddr : nullptr;
        const int group = a.gate_period ? (int)(t / a.gate_period) : 0;
        const type *gate = a.gate_period ? static_cast<const type *>(a.gate) + group * a.ldg : nullptr;
        const float rho = a.w_post ? a.rstd[t] : 1.f, rho2 = a.rstd[a.T + t];
        float r[N], h[N], u[N], dr[N], g[N];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * threads + (int)threadIdx.x) * VW;
            const bool in = c < D;
            P::unpack(in ? P::load(x + c) : P::zero(), r + v * VW);
            P::unpack(in ? P::load(y + c) : P::zero(), h + v * VW);
            P::unpack(in ? P::load(pn + c) : P::zero(), u + v * VW);
            P::unpack(in && pr ? P::load(pr + c) : P::zero(), dr + v * VW);
            if (gate) P::unpack(in ? P::load(gate + c) : P::zero(), g + v * VW);
        }
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (!gate) g[i] = 1.f;
            // h becomes y rho; r the residual sum; u = dn w_pre
            h[i] *= rho;
            r[i] = fmaf(a.scale * g[i], h[i] * w_post[i], r[i]);
            dw_pre[i] = fmaf(u[i], r[i] * rho2, dw_pre[i]);
            u[i] *= w_pre[i];
            sum = fmaf(u[i], r[i], sum);
        }
        sum = red.sum(sum) * inv_d * rho2 * rho2;
        float sum2 = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
#pragma unroll
            for (int e = 0; e < VW; ++e) {
                const int i = v * VW + e;
                const float dx = fmaf(rho2, fmaf(-r[i], sum, u[i]), dr[i]);
                r[i] = dx;
                const float dh = a.scale * dx;
                dgate[i] = fmaf(dh, h[i] * w_post[i], dgate[i]);
                u[i] = dh * g[i];
                dw_post[i] = fmaf(u[i], h[i], dw_post[i]);
                u[i] *= w_post[i];
                sum2 = fmaf(u[i], h[i], sum2);
            }
        }
        // with h = y rho: dy = rho (v - h mean(v h)); without the norm rho is 1 and dy = v
        sum2 = a.w_post ? red.sum(sum2) * inv_d : 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * threads + (int)threadIdx.x) * VW;
            if (c >= D) continue;
            P::store(static_cast<type *>(a.dx) + t * a.lddx + c, r + v * VW);
            float dy[VW];
#pragma unroll
            for (int e = 0; e < VW; ++e) {
                const int i = v * VW + e;
                dy[e] = rho * fmaf(-h[i], sum2, u[i]);
            }
            P::store(static_cast<type *>(a.dy) + t * a.lddy + c, dy);
        }
        if (gate && (t + 1 == end || (t + 1) % a.gate_period == 0)) {
            // the gate row's sum: whole when all of its rows are this block's, otherwise one
            // of the block's two partial sums (the first gate row it meets, or the last)
            const int64_t g0 = (int64_t)group * a.gate_period, g1 = g0 + a.gate_period;
            const bool whole = g0 >= begin && g1 <= end;
            const int slot = group == begin / a.gate_period ? 2 : 3;
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int e = 0; e < VW; ++e) {
                    const int c = (v * threads + (int)threadIdx.x) * VW + e, i = v * VW + e;
                    if (c < D) {
                        if (whole)
                            static_cast<type *>(a.dgate)[group * a.lddg + c] = E::from_float(dgate[i]);
                        else
                            partial[(int64_t)slot * D + c] = dgate[i];
                    }
                    dgate[i] = 0.f;
                }
        }
    }
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < VW; ++e) {
            const int c = (v * threads + (int)threadIdx.x) * VW + e, i = v * VW + e;
            if (c < D) {
                partial[c] = dw_pre[i];
                partial[D + c] = dw_post[i];
            }
        }
}

// The same for rows too wide for a block's registers: the row is read again
// for each step, and the sums over rows live in `partial`.
template <int DT>
__global__ void __launch_bounds__(1024, 1) block_norm_grad_wide_kernel(const BlockNormGradArgs a) {
    using E = Elem<DT>;
    using type = typename E::type;
    __shared__ float slots[64];
    RowReducer red{slots, (int)(blockDim.x >> 5)};
    const int D = a.D;
    const float inv_d = 1.f / (float)D;
    const int begin = block_first_row(blockIdx.x, a.T, gridDim.x);
    const int end = block_first_row(blockIdx.x + 1, a.T, gridDim.x);
    float *partial = a.partial + (int64_t)blockIdx.x * 4 * D;
    for (int c = threadIdx.x; c < D; c += blockDim.x) partial[c] = partial[D + c] = 0.f;
    for (int64_t t = begin; t < end; ++t) {
        const int group = a.gate_period ? (int)(t / a.gate_period) : 0;
        const float rho = a.w_post ? a.rstd[t] : 1.f, rho2 = a.rstd[a.T + t];
        const int64_t g0 = (int64_t)group * a.gate_period, g1 = g0 + a.gate_period;
        const bool whole = g0 >= begin && g1 <= end;
        const bool first = a.gate_period && (t == begin || t % a.gate_period == 0);
        const bool last = a.gate_period && (t + 1 == end || (t + 1) % a.gate_period == 0);
        float *gate_sum = partial + (int64_t)(a.gate_period && group == begin / a.gate_period ? 2 : 3) * D;
        struct Row {
            float h, g, w_post, r, u, dn;
        };
        auto row = [&](int c) {
            Row e;
            e.h = E::to_float(static_cast<const type *>(a.y)[t * a.ldy + c]) * rho;
            e.g = a.gate_period ? E::to_float(static_cast<const type *>(a.gate)[group * a.ldg + c]) : 1.f;
            e.w_post = a.w_post ? load_weight<DT>(a.w_post, a.w_f32, c) : 1.f;
            e.r = fmaf(a.scale * e.g, e.h * e.w_post, E::to_float(static_cast<const type *>(a.x)[t * a.ldx + c]));
            e.dn = E::to_float(static_cast<const type *>(a.dn)[t * a.lddn + c]);
            e.u = e.dn * load_weight<DT>(a.w_pre, a.w_f32, c);
            return e;
        };
        float sum = 0.f;
        for (int c = threadIdx.x; c < D; c += blockDim.x) {
            const Row e = row(c);
            sum = fmaf(e.u, e.r, sum);
        }
        sum = red.sum(sum) * inv_d * rho2 * rho2;
        auto grad_x = [&](const Row &e, int c) {
            const float dr = a.dr ? E::to_float(static_cast<const type *>(a.dr)[t * a.lddr + c]) : 0.f;
            return fmaf(rho2, fmaf(-e.r, sum, e.u), dr);
        };
        float sum2 = 0.f;
        if (a.w_post) {
            for (int c = threadIdx.x; c < D; c += blockDim.x) {
                const Row e = row(c);
                sum2 = fmaf(a.scale * grad_x(e, c) * e.g * e.w_post, e.h, sum2);
            }
            sum2 = red.sum(sum2) * inv_d;
        }
        // dx and dy may overwrite dn and dr: each element is read before the same thread writes it
        for (int c = threadIdx.x; c < D; c += blockDim.x) {
            const Row e = row(c);
            const float dx = grad_x(e, c), dh = a.scale * dx;
            partial[c] = fmaf(e.dn, e.r * rho2, partial[c]);
            partial[D + c] = fmaf(dh * e.g, e.h, partial[D + c]);
            if (a.gate_period) {
                const float s = (first ? 0.f : gate_sum[c]) + dh * e.h * e.w_post;
                gate_sum[c] = s;
                if (last && whole) static_cast<type *>(a.dgate)[group * a.lddg + c] = E::from_float(s);
            }
            static_cast<type *>(a.dx)[t * a.lddx + c] = E::from_float(dx);
            static_cast<type *>(a.dy)[t * a.lddy + c] =
                E::from_float(rho * fmaf(-e.h, sum2, dh * e.g * e.w_post));
        }
    }
}

// Adds the blocks' partial sums: blockIdx.y 0 and 1 for the weights, 2 + b for
// the gate row that block b + 1 starts inside (once, by the first such block).
// 32 columns by 8 slices of the blocks, added in slice order.
template <int DT>
__global__ void __launch_bounds__(256) block_norm_grad_join_kernel(const BlockNormGradArgs a, int blocks) {
    __shared__ float part[8][33];
    const int D = a.D, c = blockIdx.x * 32 + threadIdx.x;
    const int what = blockIdx.y;
    int b0 = 0, b1 = blocks, group = 0;
    if (what >= 2) {
        const int b = what - 1, row = block_first_row(b, a.T, blocks);
        if (row % a.gate_period == 0) return;  // block b starts a gate row of its own
        group = row / a.gate_period;
        const int64_t g0 = (int64_t)group * a.gate_period, g1 = g0 + a.gate_period;
        if (block_first_row(b - 1, a.T, blocks) > g0) return;  // an earlier block started inside it
        b0 = b - 1;
        b1 = b + 1;
        while (b1 < blocks && block_first_row(b1, a.T, blocks) < g1) ++b1;
    } else if (what == 1 && !a.w_post) {
        return;
    }
    float s = 0.f;
    if (c < D) {
        for (int b = b0 + threadIdx.y; b < b1; b += 8) {
            int slot = what;
            if (what >= 2) slot = group == block_first_row(b, a.T, blocks) / a.gate_period ? 2 : 3;
            s += a.partial[((int64_t)b * 4 + slot) * D + c];
        }
    }
    part[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < D) {
#pragma unroll
        for (int i = 1; i < 8; ++i) s += part[i][threadIdx.x];
        if (what == 0) store_weight<DT>(a.dw_pre, a.w_f32, c, s);
        else if (what == 1) store_weight<DT>(a.dw_post, a.w_f32, c, s);
        else store_weight<DT>(a.dgate, 0, (int64_t)group * a.lddg + c, s);
    }
}

}  // namespace sgemm
