// The C interface of the products with 8-bit weights: argument checks, kernel
// choice and launch.  The contract is in include/sgemm_layers.h.

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "host.h"
#include "i8_product.cuh"
#include "i8_quantize.cuh"

namespace {

using namespace sgemm;
using sgemm_host::aligned;
using sgemm_host::by_dtype;
using sgemm_host::Device;
using sgemm_host::dtype_ok;
using sgemm_host::dtype_size;
using sgemm_host::launch;
using sgemm_host::Range;

constexpr int kMaxK = 131071;  // 2^14 K < 2^31: a sum of 8-bit products fits 32 bits

template <int DT, int VW>
int launch_quantize(int M, int K, const void *x, int ldx, int8_t *q, int64_t ldq, float *s, const Device &dev,
                    cudaStream_t stream) {
    using type = typename Elem<DT>::type;
    constexpr int NV = 16 / VW;
    const int threads = std::max(1, (K + 511) / 512) * 32;  // 16 elements a thread
    const dim3 block(threads, threads == 32 ? 4 : 1);
    const int64_t groups = ((int64_t)M + block.y - 1) / block.y;
    const int64_t most = (int64_t)dev.sms * std::max(1, 2048 / (int)(block.x * block.y));
    const int q_vec = aligned(q, VW > 1 ? VW : 1) && ldq % VW == 0;
    return launch(quantize_i8_kernel<DT, VW, NV>, dim3((unsigned)std::min(groups, most)), block, 0, stream, 1, M, K,
                  static_cast<const type *>(x), (int64_t)ldx, q, ldq, s, q_vec);
}

int quantize(int M, int K, int dtype, const void *x, int ldx, int8_t *q, int64_t ldq, float *s, const Device &dev,
             cudaStream_t stream) {
    return by_dtype(dtype, [&](auto dt) {
        constexpr int DT = decltype(dt)::value, VEC = Elem<DT>::VEC;
        using type = typename Elem<DT>::type;
        if (K > 16384)
            return launch(quantize_i8_wide_kernel<DT>, dim3((unsigned)std::min(M, 2 * dev.sms)), dim3(1024), 0, stream,
                          1, M, K, static_cast<const type *>(x), (int64_t)ldx, q, ldq, s);
        const bool vec = K % VEC == 0 && aligned(x, 16) && ldx % VEC == 0;
        return vec ? launch_quantize<DT, VEC>(M, K, x, ldx, q, ldq, s, dev, stream)
                   : launch_quantize<DT, 1>(M, K, x, ldx, q, ldq, s, dev, stream);
    });
}

int product(const I8Args &p, cudaStream_t stream) {
    const dim3 grid((p.N + 63) / 64, (p.M + 63) / 64);
    const int vec_a = aligned(p.A, 16) && p.lda % 16 == 0, vec_b = aligned(p.B, 16) && p.ldb % 16 == 0;
    return launch(i8_tile_kernel, grid, dim3(256), 0, stream, 1, p, vec_a, vec_b);
}

// Rows of the quantised activations in sgemm_linear_i8's workspace.
int64_t ld16(int K) { return ((int64_t)K + 15) / 16 * 16; }

bool output_ok(int M, int N, int K, const signed char *B, int ldb, const float *b_scale, const float *bias,
               const void *C, int ldc, int ctype) {
    if (M < 0 || N < 0 || K < 0 || K > kMaxK || !dtype_ok(ctype)) return false;
    if (ldb < std::max(K, 1) || ldc < std::max(N, 1)) return false;
    if (M == 0 || N == 0) return true;
    if ((K > 0 && !B) || !b_scale || !C || !aligned(b_scale, 4) || !aligned(bias, 4)) return false;
    return aligned(C, (unsigned)dtype_size(ctype)) && (M + 63) / 64 <= 65535;
}

}  // namespace

extern "C" {

int sgemm_quantize_i8(int M, int K, int dtype, const void *x, int ldx, signed char *q, int ldq, float *s,
                      cudaStream_t stream) {
    if (M < 0 || K < 0 || !dtype_ok(dtype) || ldx < std::max(K, 1) || ldq < std::max(K, 1)) return SGEMM_ERR_INVALID_ARG;
    if (M == 0) return SGEMM_OK;
    const int size = dtype_size(dtype);
    if (!s || !aligned(s, 4) || (K > 0 && (!x || !q || !aligned(x, (unsigned)size)))) return SGEMM_ERR_INVALID_ARG;
    const Range in(x, M, K, ldx, size), out(q, M, K, ldq, 1), scale(s, 1, M, M, 4);
    if (out.overlaps(in) || scale.overlaps(in) || scale.overlaps(out)) return SGEMM_ERR_ALIAS;
    Device dev;
    if (sgemm_host::device(dev) != SGEMM_OK) return SGEMM_ERR_DEVICE;
    return quantize(M, K, dtype, x, ldx, q, ldq, s, dev, stream);
}

size_t sgemm_i8_workspace_size(int, int, int) { return 0; }

int sgemm_i8(int M, int N, int K, const signed char *A, int lda, const float *a_scale, const signed char *B, int ldb,
             const float *b_scale, const float *bias, void *C, int ldc, int ctype, void *workspace,
             size_t workspace_bytes, cudaStream_t stream) {
    if (!output_ok(M, N, K, B, ldb, b_scale, bias, C, ldc, ctype) || lda < std::max(K, 1)) return SGEMM_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return SGEMM_OK;
    if ((K > 0 && !A) || !a_scale || !aligned(a_scale, 4)) return SGEMM_ERR_INVALID_ARG;
    const size_t need = sgemm_i8_workspace_size(M, N, K);
    if (need && (!workspace || !aligned(workspace, 16) || workspace_bytes < need)) return SGEMM_ERR_INVALID_ARG;
    const Range in[5] = {Range(A, M, K, lda, 1), Range(a_scale, 1, M, M, 4), Range(B, N, K, ldb, 1),
                         Range(b_scale, 1, N, N, 4), Range(bias, 1, N, N, 4)};
    const Range c(C, M, N, ldc, dtype_size(ctype)), ws(need ? workspace : nullptr, 1, (int64_t)need, (int64_t)need, 1);
    for (const Range &i : in)
        if (c.overlaps(i) || ws.overlaps(i)) return SGEMM_ERR_ALIAS;
    if (ws.overlaps(c)) return SGEMM_ERR_ALIAS;
    Device dev;
    if (sgemm_host::device(dev) != SGEMM_OK) return SGEMM_ERR_DEVICE;
    return product(I8Args{M, N, K, A, B, lda, ldb, a_scale, b_scale, bias, C, ldc, ctype}, stream);
}

size_t sgemm_linear_i8_workspace_size(int M, int N, int K) {
    if (M <= 0 || N <= 0 || K < 0) return 0;
    return (size_t)(M * ld16(K) + ((int64_t)M + 3) / 4 * 16) + sgemm_i8_workspace_size(M, N, K);
}

int sgemm_linear_i8(int M, int N, int K, int xtype, const void *X, int ldx, const signed char *B, int ldb,
                    const float *b_scale, const float *bias, void *C, int ldc, int ctype, void *workspace,
                    size_t workspace_bytes, cudaStream_t stream) {
    if (!output_ok(M, N, K, B, ldb, b_scale, bias, C, ldc, ctype) || !dtype_ok(xtype) || ldx < std::max(K, 1))
        return SGEMM_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return SGEMM_OK;
    const int size = dtype_size(xtype);
    if (K > 0 && (!X || !aligned(X, (unsigned)size))) return SGEMM_ERR_INVALID_ARG;
    const size_t need = sgemm_linear_i8_workspace_size(M, N, K);
    if (!workspace || !aligned(workspace, 16) || workspace_bytes < need) return SGEMM_ERR_INVALID_ARG;
    const Range in[4] = {Range(X, M, K, ldx, size), Range(B, N, K, ldb, 1), Range(b_scale, 1, N, N, 4),
                         Range(bias, 1, N, N, 4)};
    const Range c(C, M, N, ldc, dtype_size(ctype)), ws(workspace, 1, (int64_t)need, (int64_t)need, 1);
    for (const Range &i : in)
        if (c.overlaps(i) || ws.overlaps(i)) return SGEMM_ERR_ALIAS;
    if (ws.overlaps(c)) return SGEMM_ERR_ALIAS;
    Device dev;
    if (sgemm_host::device(dev) != SGEMM_OK) return SGEMM_ERR_DEVICE;
    int8_t *q = static_cast<int8_t *>(workspace);
    float *s = reinterpret_cast<float *>(q + M * ld16(K));
    const int st = quantize(M, K, xtype, X, ldx, q, ld16(K), s, dev, stream);
    if (st != SGEMM_OK) return st;
    return product(I8Args{M, N, K, q, B, ld16(K), ldb, s, b_scale, bias, C, ldc, ctype}, stream);
}

}  // extern "C"
