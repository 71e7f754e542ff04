// The C interface of the row-wise operators: argument checks, kernel choice
// and launch.  The contract is in include/sgemm_layers.h.

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "block_norm.cuh"
#include "host.h"
#include "logprobs.cuh"
#include "logprobs_host.h"
#include "row_host.h"

namespace {

using namespace sgemm;
using sgemm_host::aligned;
using sgemm_host::by_dtype;
using sgemm_host::Device;
using sgemm_host::dtype_ok;
using sgemm_host::dtype_size;
using sgemm_host::launch;
using sgemm_host::kMaxWidth;
using sgemm_host::logprobs_by_length;
using sgemm_host::logprobs_shape_ok;
using sgemm_host::most_grad_runners;
using sgemm_host::Range;
using sgemm_host::row_threads;
using sgemm_host::RowPlan;
using sgemm_host::Rows;

constexpr int kMaxRows = 1 << 30;
bool finite(float v) { return std::isfinite(v); }

// ---------------------------------------------------------------- block norm

template <int DT, bool ALIGNED, int NV, int MAXT, int MINB>
int launch_norm(BlockNormArgs a, const Device &dev, cudaStream_t stream) {
    static std::atomic<int> regs[sgemm_host::kMaxDevices];
    const auto kernel = block_norm_kernel<DT, ALIGNED, NV, MAXT, MINB>;
    constexpr int size = sizeof(typename Elem<DT>::type);
    const RowPlan plan(a.D, size, kNormStages * (a.gate_period == 1 ? 3 : 2), NV * Elem<DT>::VEC, MAXT);
    a.ranks = plan.ranks;
    a.width = plan.width;
    const int fit = sgemm_host::blocks_per_sm(regs, dev, kernel, plan.threads(), (int)plan.smem);
    if (!fit) return SGEMM_ERR_LAUNCH;
    const int64_t groups = ((int64_t)a.T + plan.block.y - 1) / plan.block.y;
    const int64_t most = std::max(1, dev.sms * fit / plan.ranks);
    return launch(kernel, dim3((unsigned)(std::min(groups, most) * plan.ranks)), plan.block, plan.smem, stream,
                  (unsigned)plan.ranks, a);
}

template <int DT, bool ALIGNED>
int norm_by_width(const BlockNormArgs &a, const Device &dev, cudaStream_t stream) {
    constexpr int VEC = Elem<DT>::VEC;
    // 16 elements a thread (32768 x 1024 BF16 48 us, with 8 58): two blocks an SM while 320 threads
    // are enough (6553 x 5120 49 us, one block of up to 512 threads 69); rows of single elements,
    // whose addresses and tests take the registers, 8 while they are narrow
    if (a.D > 5120) return launch_norm<DT, ALIGNED, 16 / VEC, 512, 1>(a, dev, stream);
    if constexpr (!ALIGNED)
        if (a.D <= 2048) return launch_norm<DT, false, 8 / VEC, 256, 3>(a, dev, stream);
    return launch_norm<DT, ALIGNED, 16 / VEC, 320, ALIGNED ? 2 : 1>(a, dev, stream);
}

template <int DT, bool ALIGNED, bool TOKEN, int PER>
int launch_norm_grad(BlockNormGradArgs a, const Device &dev, cudaStream_t stream) {
    static std::atomic<int> regs[sgemm_host::kMaxDevices];
    constexpr int most = ALIGNED ? 512 : 480;  // single elements take more registers
    const auto kernel = block_norm_grad_kernel<DT, ALIGNED, PER / Elem<DT>::VEC, TOKEN, most>;
    constexpr int size = sizeof(typename Elem<DT>::type);
    const RowPlan plan(a.D, size, kNormGradStages * (3 + TOKEN + (a.dr != nullptr)), PER, most);
    a.ranks = plan.ranks;
    a.width = plan.width;
    if (!sgemm_host::blocks_per_sm(regs, dev, kernel, plan.threads(), (int)plan.smem)) return SGEMM_ERR_LAUNCH;
    const int fit = std::max(1, std::min(512 / plan.threads(), 226 * 1024 / (int)(plan.smem + 2048)));
    a.runners = std::min(most_grad_runners(a.T, a.D, dev.sms), std::max(1, dev.sms * fit / plan.ranks) * (int)plan.block.y);
    const unsigned groups = (a.runners + plan.block.y - 1) / plan.block.y;
    const int st = launch(kernel, dim3(groups * plan.ranks), plan.block, plan.smem, stream, (unsigned)plan.ranks, a);
    if (st != SGEMM_OK) return st;
    const int gates = a.gate_period > 1 ? std::min({a.T / a.gate_period, a.runners - 1, 16}) : 0;
    return launch<true>(block_norm_grad_join_kernel<DT>, dim3((a.D + 31) / 32, 2 + gates), dim3(32, kNormJoinSlices), 0, stream, 1, a);
}

template <int DT>
int norm_grad_by_layout(const BlockNormGradArgs &a, bool vec, const Device &dev, cudaStream_t stream) {
    if (a.gate_period == 1)
        return vec ? launch_norm_grad<DT, true, true, 8>(a, dev, stream) : launch_norm_grad<DT, false, true, 8>(a, dev, stream);
    // 16 elements a thread halve what a row costs beside them (8192 x 4096 BF16: 88 us with 8, 82
    // with 16); FP32, which unpacks nothing, does with 8, and 16 spill
    constexpr int PER = DT == SGEMM_F32 ? 8 : 16;
    return vec ? launch_norm_grad<DT, true, false, PER>(a, dev, stream) : launch_norm_grad<DT, false, false, 8>(a, dev, stream);
}

// Checks that the forward and the backward pass share.
bool norm_shape_ok(int T, int D, int dtype, int wdtype, const void *w_pre, const void *w_post, const Rows &gate,
                   int gate_rows, float scale) {
    if (T < 0 || D < 0 || T > kMaxRows || D > kMaxWidth || !dtype_ok(dtype)) return false;
    if (wdtype != SGEMM_F32 && wdtype != dtype) return false;
    if (!finite(scale) || gate_rows < 0) return false;
    if (T == 0 || D == 0) return true;
    const unsigned ws = dtype_size(wdtype);
    if (!w_pre || !aligned(w_pre, ws) || !aligned(w_post, ws)) return false;
    if ((gate_rows > 0) != (gate.p != nullptr)) return false;
    return !gate.p || (gate_rows <= T && T % gate_rows == 0 && gate.ok(D, dtype_size(dtype)));
}

// ---------------------------------------------------------------- log probabilities

template <int DT, int VW>
int launch_logprobs_grad(const LogprobGradArgs &a, cudaStream_t stream) {
    constexpr int THREADS = 256, U = VW > 1 ? 4 : 8;
    const unsigned cols = (unsigned)std::max(1, (a.V / VW + THREADS * U - 1) / (THREADS * U));
    const unsigned rows = (unsigned)std::min(a.T, 65535);
    const dim3 grid(cols, rows);
    if (a.mask) return launch(logprobs_grad_kernel<DT, VW, THREADS, U, true>, grid, dim3(THREADS), 0, stream, 1, a);
    return launch(logprobs_grad_kernel<DT, VW, THREADS, U, false>, grid, dim3(THREADS), 0, stream, 1, a);
}

}  // namespace

extern "C" {

int sgemm_block_norm(int T, int D, int dtype, const void *x, int ldx, const void *y, int ldy, const void *w_pre,
                     const void *w_post, int wdtype, const void *gate, int ldg, int gate_rows, float scale, float eps,
                     void *r, int ldr, void *n, int ldn, signed char *q, int ldq, float *q_scale, float *rstd,
                     cudaStream_t stream) {
    const Rows X{x, ldx}, Y{y, ldy}, G{gate, ldg}, R{r, ldr}, N{n, ldn}, Q{q, ldq};
    if (!norm_shape_ok(T, D, dtype, wdtype, w_pre, w_post, G, gate_rows, scale)) return SGEMM_ERR_INVALID_ARG;
    if (!(eps >= 0.f) || !finite(eps)) return SGEMM_ERR_INVALID_ARG;
    if (T == 0 || D == 0) return SGEMM_OK;
    const int size = dtype_size(dtype);
    if (!X.ok(D, size) || !Y.ok(D, size) || !R.ok(D, size) || (n && !N.ok(D, size)) || (!n && !q))
        return SGEMM_ERR_INVALID_ARG;
    if ((q && (!Q.ok(D, 1) || !q_scale)) || !aligned(q_scale, 4) || !aligned(rstd, 4)) return SGEMM_ERR_INVALID_ARG;

    const Range in[5] = {X.range(T, D, size), Y.range(T, D, size), G.range(gate_rows, D, size),
                         Range(w_pre, 1, D, D, dtype_size(wdtype)), Range(w_post, 1, D, D, dtype_size(wdtype))};
    const Range out[5] = {R.range(T, D, size), N.range(T, D, size), Q.range(T, D, 1), Range(q_scale, 1, q ? T : 0, T, 4),
                          Range(rstd, 2, T, T, 4)};
    for (int o = 0; o < 5; ++o) {
        for (int i = 0; i < 5; ++i)
            if (out[o].overlaps(in[i]) && !(o == 0 && i == 0 && R.same(X))) return SGEMM_ERR_ALIAS;
        for (int p = 0; p < o; ++p)
            if (out[o].overlaps(out[p])) return SGEMM_ERR_ALIAS;
    }
    Device dev;
    if (sgemm_host::device(dev) != SGEMM_OK) return SGEMM_ERR_DEVICE;
    BlockNormArgs a{T, D, x, y, gate, ldx, ldy, ldg, w_pre, w_post, wdtype == SGEMM_F32,
                    gate_rows ? T / gate_rows : 0, scale, eps, r, n, ldr, ldn, q, ldq, q_scale, rstd, 0};
    const int vec_elems = 16 / size;
    const bool vec = D % vec_elems == 0 && X.vec(size) && Y.vec(size) && G.vec(size) && R.vec(size) && N.vec(size) &&
                     aligned(w_pre, 16) && aligned(w_post, 16);
    a.q_vec = aligned(q, (unsigned)vec_elems) && ldq % vec_elems == 0;
    return by_dtype(dtype, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        return vec ? norm_by_width<DT, true>(a, dev, stream) : norm_by_width<DT, false>(a, dev, stream);
    });
}

size_t sgemm_block_norm_backward_workspace_size(int T, int D) {
    Device dev;
    if (T <= 0 || D <= 0 || sgemm_host::device(dev) != SGEMM_OK) return 0;
    return (size_t)most_grad_runners(T, D, dev.sms) * 4 * (size_t)D * sizeof(float);
}

int sgemm_block_norm_backward(int T, int D, int dtype, const void *x, int ldx, const void *y, int ldy,
                              const void *w_pre, const void *w_post, int wdtype, const void *gate, int ldg,
                              int gate_rows, float scale, const float *rstd, const void *dn, int lddn, const void *dr,
                              int lddr, void *dx, int lddx, void *dy, int lddy, void *dw_pre, void *dw_post,
                              void *dgate, int lddg, void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    const Rows X{x, ldx}, Y{y, ldy}, G{gate, ldg}, DN{dn, lddn}, DR{dr, lddr}, DX{dx, lddx}, DY{dy, lddy}, DG{dgate, lddg};
    if (!norm_shape_ok(T, D, dtype, wdtype, w_pre, w_post, G, gate_rows, scale)) return SGEMM_ERR_INVALID_ARG;
    const int size = dtype_size(dtype), wsize = dtype_size(wdtype);
    if (D == 0) return SGEMM_OK;
    if (!dw_pre || !aligned(dw_pre, (unsigned)wsize) || !aligned(dw_post, (unsigned)wsize)) return SGEMM_ERR_INVALID_ARG;
    if ((w_post != nullptr) != (dw_post != nullptr) || (gate != nullptr) != (dgate != nullptr))
        return SGEMM_ERR_INVALID_ARG;
    if (T == 0) {
        // sums over no rows; the gaps between the gate's rows stay as they are
        const bool gates = dgate && gate_rows > 0;
        if (gates && !DG.ok(D, size)) return SGEMM_ERR_INVALID_ARG;
        if (cudaMemsetAsync(dw_pre, 0, (size_t)D * wsize, stream) != cudaSuccess ||
            (dw_post && cudaMemsetAsync(dw_post, 0, (size_t)D * wsize, stream) != cudaSuccess) ||
            (gates && cudaMemset2DAsync(dgate, (size_t)lddg * size, 0, (size_t)D * size, (size_t)gate_rows, stream) != cudaSuccess)) {
            (void)cudaGetLastError();
            return SGEMM_ERR_LAUNCH;
        }
        return SGEMM_OK;
    }
    if (!X.ok(D, size) || !Y.ok(D, size) || !DN.ok(D, size) || (dr && !DR.ok(D, size)) || !DX.ok(D, size) ||
        !DY.ok(D, size) || (dgate && !DG.ok(D, size)) || !rstd || !aligned(rstd, 4))
        return SGEMM_ERR_INVALID_ARG;
    Device dev;
    if (sgemm_host::device(dev) != SGEMM_OK) return SGEMM_ERR_DEVICE;
    const size_t need = sgemm_block_norm_backward_workspace_size(T, D);
    if (!workspace || !aligned(workspace, 16) || workspace_bytes < need) return SGEMM_ERR_INVALID_ARG;

    const Range in[8] = {DN.range(T, D, size), DR.range(T, D, size), X.range(T, D, size), Y.range(T, D, size),
                         G.range(gate_rows, D, size), Range(w_pre, 1, D, D, wsize), Range(w_post, 1, D, D, wsize),
                         Range(rstd, 2, T, T, 4)};
    const Range out[6] = {DX.range(T, D, size), DY.range(T, D, size), DG.range(gate_rows, D, size),
                          Range(dw_pre, 1, D, D, wsize), Range(dw_post, 1, D, D, wsize),
                          Range(workspace, 1, (int64_t)need, (int64_t)need, 1)};
    const Rows *outs[2] = {&DX, &DY}, *ins[2] = {&DN, &DR};
    for (int o = 0; o < 6; ++o) {
        for (int i = 0; i < 8; ++i)
            if (out[o].overlaps(in[i]) && !(o < 2 && i < 2 && outs[o]->same(*ins[i]))) return SGEMM_ERR_ALIAS;
        for (int p = 0; p < o; ++p)
            if (out[o].overlaps(out[p])) return SGEMM_ERR_ALIAS;
    }
    const BlockNormGradArgs a{T, D, x, y, gate, dn, dr, ldx, ldy, ldg, lddn, lddr, w_pre, w_post, wdtype == SGEMM_F32,
                              gate_rows ? T / gate_rows : 0, scale, rstd, dx, dy, dgate, lddx, lddy, lddg, dw_pre,
                              dw_post, static_cast<float *>(workspace), 0};
    const bool vec = D % (16 / size) == 0 && X.vec(size) && Y.vec(size) && G.vec(size) && DN.vec(size) &&
                     DR.vec(size) && DX.vec(size) && DY.vec(size) && DG.vec(size) && aligned(w_pre, 16) &&
                     aligned(w_post, 16);
    return by_dtype(dtype, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        return norm_grad_by_layout<DT>(a, vec, dev, stream);
    });
}

int sgemm_logprobs(int T, int V, int dtype, const void *logits, int ldz, float scale, const int32_t *mask, int ldm,
                   int mask_rows, const int64_t *target, float *logprob, float *entropy, float *lse, int top,
                   float *top_logprob, int32_t *top_id, cudaStream_t stream) {
    const Rows Z{logits, ldz};
    if (!logprobs_shape_ok(T, V, dtype, Z, scale, mask, ldm, mask_rows)) return SGEMM_ERR_INVALID_ARG;
    if (top < 0 || top > 32) return SGEMM_ERR_INVALID_ARG;
    if (T == 0) return SGEMM_OK;
    if ((top > 0 && (!top_logprob || !top_id)) || (logprob && !target)) return SGEMM_ERR_INVALID_ARG;
    if (!aligned(target, 8) || !aligned(logprob, 4) || !aligned(entropy, 4) || !aligned(lse, 4) ||
        !aligned(top_logprob, 4) || !aligned(top_id, 4))
        return SGEMM_ERR_INVALID_ARG;
    const int words = (V + 31) / 32;
    const Range in[3] = {Z.range(T, V, dtype_size(dtype)), Range(mask, mask_rows, words, ldm, 4), Range(target, 1, T, T, 8)};
    const Range out[5] = {Range(logprob, 1, T, T, 4), Range(entropy, 1, T, T, 4), Range(lse, 1, T, T, 4),
                          Range(top ? top_logprob : nullptr, T, top, top, 4), Range(top ? top_id : nullptr, T, top, top, 4)};
    for (int o = 0; o < 5; ++o) {
        for (const Range &i : in)
            if (out[o].overlaps(i)) return SGEMM_ERR_ALIAS;
        for (int p = 0; p < o; ++p)
            if (out[o].overlaps(out[p])) return SGEMM_ERR_ALIAS;
    }
    Device dev;
    if (sgemm_host::device(dev) != SGEMM_OK) return SGEMM_ERR_DEVICE;
    const LogprobArgs a{T, V, logits, ldz, scale, mask, mask_rows > 1 ? ldm : 0, target, logprob, entropy, lse, top,
                        top_logprob, top_id, nullptr, nullptr, nullptr};
    return by_dtype(dtype, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        return mask ? logprobs_by_length<DT, true, false>(a, dev, stream) : logprobs_by_length<DT, false, false>(a, dev, stream);
    });
}

int sgemm_logprobs_backward(int T, int V, int dtype, const void *logits, int ldz, float scale, const int32_t *mask,
                            int ldm, int mask_rows, const int64_t *target, const float *lse, const float *entropy,
                            const float *g_logprob, const float *g_entropy, void *dz, int lddz, cudaStream_t stream) {
    const Rows Z{logits, ldz}, DZ{dz, lddz};
    if (!logprobs_shape_ok(T, V, dtype, Z, scale, mask, ldm, mask_rows)) return SGEMM_ERR_INVALID_ARG;
    if (T == 0 || V == 0) return SGEMM_OK;
    const int size = dtype_size(dtype);
    if (!DZ.ok(V, size) || !target || !lse || !g_logprob || (g_entropy && !entropy)) return SGEMM_ERR_INVALID_ARG;
    if (!aligned(target, 8) || !aligned(lse, 4) || !aligned(entropy, 4) || !aligned(g_logprob, 4) || !aligned(g_entropy, 4))
        return SGEMM_ERR_INVALID_ARG;
    const int words = (V + 31) / 32;
    const Range out = DZ.range(T, V, size);
    const Range in[6] = {Range(mask, mask_rows, words, ldm, 4), Range(target, 1, T, T, 8), Range(lse, 1, T, T, 4),
                         Range(entropy, 1, T, T, 4), Range(g_logprob, 1, T, T, 4), Range(g_entropy, 1, T, T, 4)};
    for (const Range &i : in)
        if (out.overlaps(i)) return SGEMM_ERR_ALIAS;
    if (out.overlaps(Z.range(T, V, size)) && !DZ.same(Z)) return SGEMM_ERR_ALIAS;
    const LogprobGradArgs a{T, V, logits, ldz, scale, mask, mask_rows > 1 ? ldm : 0, target, lse, entropy, g_logprob,
                            g_entropy, dz, lddz};
    // 16-byte pieces where z and dz are at the same distance from a 16-byte boundary in every row
    const bool vec = (reinterpret_cast<uintptr_t>(logits) & 15u) == (reinterpret_cast<uintptr_t>(dz) & 15u) &&
                     (T == 1 || ((int64_t)ldz - lddz) * size % 16 == 0);
    return by_dtype(dtype, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        return vec ? launch_logprobs_grad<DT, Elem<DT>::VEC>(a, stream) : launch_logprobs_grad<DT, 1>(a, stream);
    });
}

}  // extern "C"
