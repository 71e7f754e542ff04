// The C interface of the layer norm: argument checks, kernel choice and launch.
// The contract is in include/sgemm_layers.h.

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "host.h"
#include "layer_norm.cuh"
#include "row_host.h"

namespace {

using namespace sgemm;
using sgemm_host::aligned;
using sgemm_host::by_dtype;
using sgemm_host::Device;
using sgemm_host::dtype_ok;
using sgemm_host::dtype_size;
using sgemm_host::launch;
using sgemm_host::Range;
using sgemm_host::RowPlan;
using sgemm_host::Rows;

constexpr int kMaxRows = 1 << 30;

template <int DT, bool ALIGNED, int NV, int MAXT, int MINB>
int launch_norm(LayerNormArgs a, const Device &dev, cudaStream_t stream) {
    static std::atomic<int> regs[sgemm_host::kMaxDevices];
    const auto kernel = layer_norm_kernel<DT, ALIGNED, NV, MAXT, MINB>;
    constexpr int size = sizeof(typename Elem<DT>::type);
    const RowPlan plan(a.D, size, kLayerNormStages * (a.add ? 2 : 1), NV * Elem<DT>::VEC, MAXT);
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
int norm_by_width(const LayerNormArgs &a, const Device &dev, cudaStream_t stream) {
    constexpr int VEC = Elem<DT>::VEC;
    // 16 elements a thread, and two blocks an SM while 320 threads are enough (rows of single elements
    // too: 3907 x 5119 BF16 54 us, with one block 62, with 640 threads of 8 elements 58)
    // one piece a lane where a warp's are enough (64000 x 128 BF16 with a sum 19.1 us, with two 25.3)
    if (a.D <= 32 * VEC) return launch_norm<DT, ALIGNED, 1, 128, 6>(a, dev, stream);
    if (a.D > 5120) return launch_norm<DT, ALIGNED, 16 / VEC, 512, 1>(a, dev, stream);
    return launch_norm<DT, ALIGNED, 16 / VEC, 320, 2>(a, dev, stream);
}

template <int DT, bool ALIGNED, int PER, int MAXT>
int launch_norm_grad(LayerNormGradArgs a, const Device &dev, cudaStream_t stream) {
    static std::atomic<int> regs[sgemm_host::kMaxDevices];
    const auto kernel = layer_norm_grad_kernel<DT, ALIGNED, PER / Elem<DT>::VEC, MAXT>;
    constexpr int size = sizeof(typename Elem<DT>::type);
    const RowPlan plan(a.D, size, kLayerNormGradStages * (a.dr ? 3 : 2), PER, MAXT);
    a.ranks = plan.ranks;
    a.width = plan.width;
    const int held = sgemm_host::blocks_per_sm(regs, dev, kernel, plan.threads(), (int)plan.smem);
    if (!held) return SGEMM_ERR_LAUNCH;
    const int fit = std::max(1, std::min(512 / plan.threads(), held));  // (the workspace has room for no more)
    a.runners = std::min(sgemm_host::most_grad_runners(a.T, a.D, dev.sms),
                         std::max(1, dev.sms * fit / plan.ranks) * (int)plan.block.y);
    const unsigned groups = (a.runners + plan.block.y - 1) / plan.block.y;
    a.partials = (int)groups;
    const int st = launch(kernel, dim3(groups * plan.ranks), plan.block, plan.smem, stream, (unsigned)plan.ranks, a);
    if (st != SGEMM_OK) return st;
    return launch<true>(layer_norm_grad_join_kernel<DT>, dim3((a.D + 31) / 32, a.db ? 2 : 1), dim3(32, kLayerNormJoinSlices), 0,
                        stream, 1, a);
}

// The most partial sums that the gradient writes, whatever the type and the alignment: one a block, of
// which rows that every type gives to a warp have four runners each, and elsewhere one a runner.
int64_t most_grad_partials(int T, int D, int sms) {
    const int runners = sgemm_host::most_grad_runners(T, D, sms);
    return D <= 256 ? (runners + 3) / 4 : runners;
}

// Checks that the forward and the backward pass share.
bool norm_shape_ok(int T, int D, int dtype, int wdtype, const void *w) {
    if (T < 0 || D < 0 || T > kMaxRows || D > sgemm_host::kMaxWidth || !dtype_ok(dtype)) return false;
    if (wdtype != SGEMM_F32 && wdtype != dtype) return false;
    return T == 0 || D == 0 || (w && aligned(w, (unsigned)dtype_size(wdtype)));
}

}  // namespace

extern "C" {

int sgemm_layer_norm(int T, int D, int dtype, const void *x, int ldx, const void *add, int lda, const void *w, const void *b,
                     int wdtype, float eps, void *r, int ldr, void *n, int ldn, float *stats, cudaStream_t stream) {
    const Rows X{x, ldx}, A{add, lda}, R{r, ldr}, N{n, ldn};
    if (!norm_shape_ok(T, D, dtype, wdtype, w) || !(eps >= 0.f) || !std::isfinite(eps)) return SGEMM_ERR_INVALID_ARG;
    if (T == 0 || D == 0) return SGEMM_OK;
    const int size = dtype_size(dtype), wsize = dtype_size(wdtype);
    if (!X.ok(D, size) || !N.ok(D, size) || (add && !A.ok(D, size)) || (add != nullptr) != (r != nullptr) || (r && !R.ok(D, size)))
        return SGEMM_ERR_INVALID_ARG;
    if (!aligned(b, (unsigned)wsize) || !aligned(stats, 4)) return SGEMM_ERR_INVALID_ARG;
    const Range in[4] = {X.range(T, D, size), A.range(T, D, size), Range(w, 1, D, D, wsize), Range(b, 1, D, D, wsize)};
    const Range out[3] = {R.range(T, D, size), N.range(T, D, size), Range(stats, 2, T, T, 4)};
    for (int o = 0; o < 3; ++o) {
        for (int i = 0; i < 4; ++i)
            if (out[o].overlaps(in[i]) && !(o == 0 && ((i == 0 && R.same(X)) || (i == 1 && R.same(A))))) return SGEMM_ERR_ALIAS;
        for (int p = 0; p < o; ++p)
            if (out[o].overlaps(out[p])) return SGEMM_ERR_ALIAS;
    }
    Device dev;
    if (sgemm_host::device(dev) != SGEMM_OK) return SGEMM_ERR_DEVICE;
    const LayerNormArgs a{T, D, x, add, ldx, lda, w, b, wdtype == SGEMM_F32, eps, r, n, ldr, ldn, stats, 1, D};
    const bool vec = D % (16 / size) == 0 && X.vec(size) && A.vec(size) && R.vec(size) && N.vec(size) && aligned(w, 16) &&
                     aligned(b, 16);
    return by_dtype(dtype, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        return vec ? norm_by_width<DT, true>(a, dev, stream) : norm_by_width<DT, false>(a, dev, stream);
    });
}

size_t sgemm_layer_norm_backward_workspace_size(int T, int D) {
    Device dev;
    if (T <= 0 || D <= 0 || T > kMaxRows || D > sgemm_host::kMaxWidth || sgemm_host::device(dev) != SGEMM_OK) return 0;
    return (size_t)most_grad_partials(T, D, dev.sms) * 2 * (size_t)D * sizeof(float);
}

int sgemm_layer_norm_backward(int T, int D, int dtype, const void *x, int ldx, const void *w, int wdtype, const float *stats,
                              const void *dn, int lddn, const void *dr, int lddr, void *dx, int lddx, void *dw, void *db,
                              void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    const Rows X{x, ldx}, DN{dn, lddn}, DR{dr, lddr}, DX{dx, lddx};
    if (!norm_shape_ok(T, D, dtype, wdtype, w)) return SGEMM_ERR_INVALID_ARG;
    if (D == 0) return SGEMM_OK;
    const int size = dtype_size(dtype), wsize = dtype_size(wdtype);
    if (!dw || !aligned(dw, (unsigned)wsize) || !aligned(db, (unsigned)wsize)) return SGEMM_ERR_INVALID_ARG;
    if (T == 0) {
        // sums over no rows
        if (Range(dw, 1, D, D, wsize).overlaps(Range(db, 1, D, D, wsize))) return SGEMM_ERR_ALIAS;
        if (cudaMemsetAsync(dw, 0, (size_t)D * wsize, stream) != cudaSuccess ||
            (db && cudaMemsetAsync(db, 0, (size_t)D * wsize, stream) != cudaSuccess)) {
            (void)cudaGetLastError();
            return SGEMM_ERR_LAUNCH;
        }
        return SGEMM_OK;
    }
    if (!X.ok(D, size) || !DN.ok(D, size) || (dr && !DR.ok(D, size)) || !DX.ok(D, size) || !stats || !aligned(stats, 4))
        return SGEMM_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 16)) return SGEMM_ERR_INVALID_ARG;
    // the workspace's size, which depends on the device, is checked last
    const Range in[5] = {DN.range(T, D, size), DR.range(T, D, size), X.range(T, D, size), Range(w, 1, D, D, wsize),
                         Range(stats, 2, T, T, 4)};
    const Rows *ins[3] = {&DN, &DR, &X};
    auto clear = [&](const Range (&out)[4]) {
        for (int o = 0; o < 4; ++o) {
            for (int i = 0; i < 5; ++i)
                if (out[o].overlaps(in[i]) && !(o == 0 && i < 3 && DX.same(*ins[i]))) return false;
            for (int p = 0; p < o; ++p)
                if (out[o].overlaps(out[p])) return false;
        }
        return true;
    };
    const Range outs[3] = {DX.range(T, D, size), Range(dw, 1, D, D, wsize), Range(db, 1, D, D, wsize)};
    if (!clear({outs[0], outs[1], outs[2], Range()})) return SGEMM_ERR_ALIAS;
    Device dev;
    if (sgemm_host::device(dev) != SGEMM_OK) return SGEMM_ERR_DEVICE;
    const size_t need = sgemm_layer_norm_backward_workspace_size(T, D);
    if (workspace_bytes < need) return SGEMM_ERR_INVALID_ARG;
    if (!clear({outs[0], outs[1], outs[2], Range(workspace, 1, (int64_t)need, (int64_t)need, 1)})) return SGEMM_ERR_ALIAS;
    const LayerNormGradArgs a{T, D, x, dn, dr, ldx, lddn, lddr, w, wdtype == SGEMM_F32, stats, dx, lddx, dw, db,
                              static_cast<float *>(workspace), 0, 0, 1, D};
    const bool vec = D % (16 / size) == 0 && X.vec(size) && DN.vec(size) && DR.vec(size) && DX.vec(size) && aligned(w, 16);
    return by_dtype(dtype, [&](auto dt) {
        // 16-bit rows of single elements: 320 threads of 16, which take more registers (6664 x 3001 BF16
        // 47.6 us, with 8 elements 59.5; 3907 x 5119, where those are a cluster's, 55 and 106)
        constexpr int DT = decltype(dt)::value, PER = DT == SGEMM_F32 ? 8 : 16, ONE = Elem<DT>::VEC;
        // one piece a lane where a warp's are enough (64000 x 128 BF16 with dr 22.1 us, with two 28.3)
        if (D <= 32 * ONE)
            return vec ? launch_norm_grad<DT, true, ONE, 128>(a, dev, stream) : launch_norm_grad<DT, false, ONE, 128>(a, dev, stream);
        // FP32 rows that 8 elements a thread would share out over a cluster: 16 elements, which keep them within
        // fewer blocks (2000 x 5120 with dr 32 us, with 8 53), or where three inputs of a row fill the ring sooner
        // within as many (x 8192 64.6 and 65.0, x 12800 192 and 201).  Rows of single elements: where there are
        // fewer blocks (x 8191 91 and 136; but x 16383 323 and 284), or where 192 threads leave room for a second
        // block an SM (x 6001 57 and 76, x 11001 165 and 266; with 224 threads x 7167 87 and 81).
        if constexpr (DT == SGEMM_F32) {
            const int slots = kLayerNormGradStages * (dr ? 3 : 2);
            const RowPlan wide(D, size, slots, 16, 320), narrow(D, size, slots, 8, 480);
            if (vec ? D > 8 * 512 : narrow.ranks > 1 && (wide.ranks < narrow.ranks || wide.threads() <= 192))
                return vec ? launch_norm_grad<DT, true, 16, 512>(a, dev, stream) : launch_norm_grad<DT, false, 16, 320>(a, dev, stream);
        }
        return vec ? launch_norm_grad<DT, true, PER, 512>(a, dev, stream)
                   : launch_norm_grad<DT, false, PER, DT == SGEMM_F32 ? 480 : 320>(a, dev, stream);
    });
}

}  // extern "C"
