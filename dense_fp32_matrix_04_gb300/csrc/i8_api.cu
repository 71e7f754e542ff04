// The C interface of the products with 8-bit weights: argument checks, kernel
// choice and launch.  The contract is in include/sgemm_layers.h.

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "host.h"
#include "i8_decode.cuh"
#include "i8_quantize.cuh"
#include "i8_tcgen05.cuh"

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

// Codes as 8-bit integers (Code int8_t) or as FP16 values on padded rows (__half).
template <int DT, int VW, class Code>
int launch_quantize(int M, int K, const void *x, int ldx, Code *q, int64_t ldq, float *s, const Device &dev,
                    cudaStream_t stream) {
    using type = typename Elem<DT>::type;
    constexpr int NV = 16 / VW;
    const int threads = std::max(1, (K + 511) / 512) * 32;  // 16 elements a thread
    const dim3 block(threads, threads == 32 ? 4 : 1);
    const int64_t groups = ((int64_t)M + block.y - 1) / block.y;
    const int64_t most = (int64_t)dev.sms * std::max(1, 2048 / (int)(block.x * block.y));
    const int q_vec = aligned(q, VW > 1 ? VW : 1) && ldq % VW == 0;
    return launch(quantize_i8_kernel<DT, VW, NV, Code>, dim3((unsigned)std::min(groups, most)), block, 0, stream, 1, M,
                  K, static_cast<const type *>(x), (int64_t)ldx, q, ldq, s, q_vec);
}

template <class Code>
int quantize(int M, int K, int dtype, const void *x, int ldx, Code *q, int64_t ldq, float *s, const Device &dev,
             cudaStream_t stream) {
    return by_dtype(dtype, [&](auto dt) {
        constexpr int DT = decltype(dt)::value, VEC = Elem<DT>::VEC;
        using type = typename Elem<DT>::type;
        if (K > 16384)
            return launch(quantize_i8_wide_kernel<DT, Code>, dim3((unsigned)std::min(M, 2 * dev.sms)), dim3(1024), 0,
                          stream, 1, M, K, static_cast<const type *>(x), (int64_t)ldx, q, ldq, s);
        const bool vec = K % VEC == 0 && aligned(x, 16) && ldx % VEC == 0;
        return vec ? launch_quantize<DT, VEC>(M, K, x, ldx, q, ldq, s, dev, stream)
                   : launch_quantize<DT, 1>(M, K, x, ldx, q, ldq, s, dev, stream);
    });
}

// Rows of 8-bit integers that start on 16 bytes.
bool rows16(const int8_t *p, int64_t ld) { return aligned(p, 16) && ld % 16 == 0; }

// ---------------------------------------------------------------- few rows of A

constexpr int kDecodeRows = 64;

template <class T, bool EARLY, bool AA, bool AB>
int launch_decode(const I8Args &p, const Device &dev, cudaStream_t stream) {
    static std::atomic<int> regs[sgemm_host::kMaxDevices];
    const auto kernel = i8_decode_kernel<T, AA, AB>;
    if (!sgemm_host::blocks_per_sm(regs, dev, kernel, T::THREADS, T::SMEM)) return SGEMM_ERR_LAUNCH;
    const int tiles = (p.N + T::ROWS - 1) / T::ROWS;
    // few rows of B: clusters of up to 8 blocks share k, while each keeps 512 of it
    unsigned ranks = 1;
    while (ranks < 8 && (int64_t)tiles * ranks < 2 * dev.sms && p.K / (int)(ranks * 2) >= 512) ranks *= 2;
    return launch<EARLY>(kernel, dim3(tiles * ranks), dim3(T::THREADS), T::SMEM, stream, ranks, p, (int)ranks);
}

template <bool EARLY, bool AA, bool AB>
int decode_by_rows(const I8Args &p, const Device &dev, cudaStream_t stream) {
    if (p.M <= 8) return launch_decode<I8DecodeTile<1, 1, 8>, EARLY, AA, AB>(p, dev, stream);
    if (p.M <= 16) return launch_decode<I8DecodeTile<1, 2, 4>, EARLY, AA, AB>(p, dev, stream);
    if (p.M <= 32) return launch_decode<I8DecodeTile<2, 4, 2>, EARLY, AA, AB>(p, dev, stream);
    return launch_decode<I8DecodeTile<2, 8, 2>, EARLY, AA, AB>(p, dev, stream);
}

// EARLY: A comes from the kernel launched just before, which B does not.
template <bool EARLY>
int decode(const I8Args &p, const Device &dev, cudaStream_t stream) {
    const bool aa = EARLY || rows16(p.A, p.lda), ab = rows16(p.B, p.ldb);
    if constexpr (!EARLY) {
        if (!aa) return ab ? decode_by_rows<false, false, true>(p, dev, stream) : decode_by_rows<false, false, false>(p, dev, stream);
    }
    return ab ? decode_by_rows<EARLY, true, true>(p, dev, stream) : decode_by_rows<EARLY, true, false>(p, dev, stream);
}

// ---------------------------------------------------------------- many rows of A

int64_t ld8(int K) { return ((int64_t)K + 7) / 8 * 8; }
int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }

// Tile width and k-splits of a product: the smallest estimate of rounds over
// the SMs times the length of one, in cycles of the tensor cores.
struct GemmPlan {
    int bn = 256, splits = 1;
    GemmPlan(int M, int N, int K, int sms) {
        const int steps = (K + 63) / 64;
        double best = 1e300;
        for (int width : {256, 128, 64}) {
            const int64_t tiles = (int64_t)((M + 127) / 128) * ((N + width - 1) / width);
            const double step = width == 256 ? 560 : width == 128 ? 320 : 220;
            for (int s = 1; s <= 16 && s <= (steps + 3) / 4; ++s) {
                const int64_t rounds = (tiles * s + sms - 1) / sms;
                double t = (double)rounds * (((steps + s - 1) / s) * step) + 1500 + width * 4;
                if (s > 1) t += 4000 + (double)s * M * N * 8 / 3000;  // the slabs out and in again, and a launch
                if (t < best) best = t, bn = width, splits = s;
            }
        }
    }
    int64_t ldp(int N) const { return ((int64_t)N + 3) / 4 * 4; }
    int64_t partial_bytes(int M, int N) const { return splits > 1 ? (int64_t)splits * M * ldp(N) * 4 : 0; }
};

template <int BN, int CT>
int launch_gemm(const I8Args &p, const __half *a, const __half *b, const GemmPlan &plan, float *partials, int vec,
                const Device &dev, cudaStream_t stream) {
    using T = I8Tile<BN>;
    static std::atomic<int> regs[sgemm_host::kMaxDevices];
    const auto kernel = i8_tcgen05_kernel<BN, CT>;
    if (!sgemm_host::blocks_per_sm(regs, dev, kernel, T::THREADS, T::SMEM_BYTES)) return SGEMM_ERR_LAUNCH;
    CUtensorMap ta, tb;
    if (!sgemm_host::encode_f16(&ta, a, p.M, p.K, ld8(p.K), T::BM) ||
        !sgemm_host::encode_f16(&tb, b, p.N, p.K, ld8(p.K), BN))
        return SGEMM_ERR_LAUNCH;
    const int64_t units = (int64_t)((p.M + T::BM - 1) / T::BM) * ((p.N + BN - 1) / BN) * plan.splits;
    return launch<true>(kernel, dim3((unsigned)std::min<int64_t>(units, dev.sms)), dim3(T::THREADS), T::SMEM_BYTES,
                        stream, 1, ta, tb, p, plan.splits, partials, plan.ldp(p.N), vec, dev.err_word,
                        sgemm_host::wait_limit_ns(), sgemm_host::test_flags());
}

template <int CT>
int gemm_by_width(const I8Args &p, const __half *a, const __half *b, const GemmPlan &plan, float *partials, int vec,
                  const Device &dev, cudaStream_t stream) {
    switch (plan.bn) {
        case 64: return launch_gemm<64, CT>(p, a, b, plan, partials, vec, dev, stream);
        case 128: return launch_gemm<128, CT>(p, a, b, plan, partials, vec, dev, stream);
        default: return launch_gemm<256, CT>(p, a, b, plan, partials, vec, dev, stream);
    }
}

// EARLY: beside the kernel before, which neither reads nor writes these.
template <bool EARLY>
int expand(int rows, int K, const int8_t *q, int64_t ldq, __half *h, const Device &dev, cudaStream_t stream) {
    const int64_t pieces = (int64_t)rows * ((K + 15) / 16);
    const dim3 grid((unsigned)std::min<int64_t>((pieces + 255) / 256, (int64_t)dev.sms * 8));
    return rows16(q, ldq) ? launch<EARLY>(i8_expand_kernel<true>, grid, dim3(256), 0, stream, 1, rows, K, q, ldq, h, ld8(K))
                          : launch<EARLY>(i8_expand_kernel<false>, grid, dim3(256), 0, stream, 1, rows, K, q, ldq, h, ld8(K));
}

int join(const I8Args &p, int splits, const float *partials, int64_t ldp, const Device &dev, cudaStream_t stream) {
    const int64_t blocks = std::min<int64_t>(((int64_t)p.M * p.N + 255) / 256, (int64_t)dev.sms * 8);
    return launch(i8_join_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, 1, p, splits, partials, ldp);
}

// The product of FP16 codes a (M x K) with the rows of p.B, which are expanded
// into b first; both on rows of ld8(K).
int gemm(const I8Args &p, const __half *a, __half *b, float *partials, const GemmPlan &plan, const Device &dev,
         cudaStream_t stream) {
    int st = expand<true>(p.N, p.K, p.B, p.ldb, b, dev, stream);
    if (st != SGEMM_OK) return st;
    if (plan.splits > 1) {
        st = gemm_by_width<SGEMM_F32>(p, a, b, plan, partials, 1, dev, stream);
        return st == SGEMM_OK ? join(p, plan.splits, partials, plan.ldp(p.N), dev, stream) : st;
    }
    const int vec = aligned(p.C, 16) && p.ldc * dtype_size(p.ctype) % 16 == 0;
    return by_dtype(p.ctype, [&](auto ct) {
        return gemm_by_width<decltype(ct)::value>(p, a, b, plan, nullptr, vec, dev, stream);
    });
}

// Bytes of the FP16 operands and of the k-splits' partial sums.
int64_t gemm_workspace(int M, int N, int K, int sms) {
    return up256(2 * M * ld8(K)) + up256(2 * N * ld8(K)) + GemmPlan(M, N, K, sms).partial_bytes(M, N);
}

int device_sms() {
    Device dev;
    return sgemm_host::device(dev) == SGEMM_OK ? dev.sms : 0;
}

// Rows of the quantised activations in sgemm_linear_i8's workspace.
int64_t ld16(int K) { return ((int64_t)K + 15) / 16 * 16; }

bool output_ok(int M, int N, int K, const signed char *B, int ldb, const float *b_scale, const float *bias,
               const void *C, int ldc, int ctype) {
    if (M < 0 || N < 0 || K < 0 || K > kMaxK || !dtype_ok(ctype)) return false;
    if (ldb < std::max(K, 1) || ldc < std::max(N, 1)) return false;
    if (M == 0 || N == 0) return true;
    if ((K > 0 && !B) || !b_scale || !C || !aligned(b_scale, 4) || !aligned(bias, 4)) return false;
    return aligned(C, (unsigned)dtype_size(ctype));
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

size_t sgemm_i8_workspace_size(int M, int N, int K) {
    if (M <= kDecodeRows || N <= 0 || K <= 0) return 0;
    const int sms = device_sms();
    return sms ? (size_t)gemm_workspace(M, N, K, sms) : 0;
}

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
    const I8Args p{M, N, K, A, B, lda, ldb, a_scale, b_scale, bias, C, ldc, ctype};
    if (K == 0) return join(p, 0, nullptr, 0, dev, stream);
    if (M <= kDecodeRows) return decode<false>(p, dev, stream);
    __half *a = static_cast<__half *>(workspace), *b = a + up256(2 * M * ld8(K)) / 2;
    float *partials = reinterpret_cast<float *>(b + up256(2 * N * ld8(K)) / 2);
    const int st = expand<false>(M, K, A, lda, a, dev, stream);
    return st == SGEMM_OK ? gemm(p, a, b, partials, GemmPlan(M, N, K, dev.sms), dev, stream) : st;
}

size_t sgemm_linear_i8_workspace_size(int M, int N, int K) {
    if (M <= 0 || N <= 0 || K < 0) return 0;
    const int64_t scales = up256(4 * (int64_t)M);
    if (M <= kDecodeRows || K == 0) return (size_t)(scales + M * ld16(K));
    const int sms = device_sms();
    return sms ? (size_t)(scales + gemm_workspace(M, N, K, sms)) : 0;
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
    float *s = static_cast<float *>(workspace);
    unsigned char *rest = static_cast<unsigned char *>(workspace) + up256(4 * (int64_t)M);
    I8Args p{M, N, K, nullptr, B, 0, ldb, s, b_scale, bias, C, ldc, ctype};
    if (M <= kDecodeRows || K == 0) {
        int8_t *q = reinterpret_cast<int8_t *>(rest);
        const int st = quantize(M, K, xtype, X, ldx, q, ld16(K), s, dev, stream);
        if (st != SGEMM_OK) return st;
        p.A = q;
        p.lda = ld16(K);
        return K == 0 ? join(p, 0, nullptr, 0, dev, stream) : decode<true>(p, dev, stream);
    }
    __half *a = reinterpret_cast<__half *>(rest), *b = a + up256(2 * M * ld8(K)) / 2;
    float *partials = reinterpret_cast<float *>(b + up256(2 * N * ld8(K)) / 2);
    const int st = quantize(M, K, xtype, X, ldx, a, ld8(K), s, dev, stream);
    return st == SGEMM_OK ? gemm(p, a, b, partials, GemmPlan(M, N, K, dev.sms), dev, stream) : st;
}

}  // extern "C"
