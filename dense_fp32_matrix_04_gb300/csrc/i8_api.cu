// The C interface of the products with 8-bit weights: argument checks, kernel
// choice and launch.  The contract is in include/sgemm_layers.h.

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "host.h"
#include "i8_quantize.cuh"
#include "i8_rows.cuh"
#include "i8_stream.cuh"

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
constexpr int kMaxRows = 1 << 30;  // of tokens and of weights: the kernels' row numbers and a round of them fit 32 bits

// Codes as 8-bit integers (Code int8_t) or as FP16 values on padded rows (__half).
template <int DT, int VW, class Code>
int launch_quantize(int M, int K, const void *x, int ldx, Code *q, int64_t ldq, float *s, const Device &dev,
                    cudaStream_t stream) {
    using type = typename Elem<DT>::type;
    constexpr int NV = 16 / VW;
    const int threads = std::max(1, (K + 511) / 512) * 32;  // 16 elements a thread
    const dim3 block(threads, threads == 32 ? 4 : 1);
    const int64_t groups = ((int64_t)M + block.y - 1) / block.y;
    static std::atomic<int> regs[sgemm_host::kMaxDevices];
    const int fit = sgemm_host::blocks_per_sm(regs, dev, quantize_i8_kernel<DT, VW, NV, Code>, (int)(block.x * block.y), 0);
    if (!fit) return SGEMM_ERR_LAUNCH;
    const int64_t most = (int64_t)dev.sms * fit;
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

int64_t ld16(int K) { return ((int64_t)K + 15) / 16 * 16; }
int64_t ld8(int K) { return ((int64_t)K + 7) / 8 * 8; }
int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }

// ---------------------------------------------------------------- up to four tokens

// Up to four tokens go to the kernel that reads whole rows, whatever K.
bool takes_rows(int M, int K) { return M <= kRowsTokens && K > 0; }

template <int MT, int XT, bool ALIGNED, int THREADS>
int launch_rows(const I8Args &p, const void *X, int64_t ldx, int smem, const Device &dev, cudaStream_t stream) {
    static std::atomic<int> regs[sgemm_host::kMaxDevices];
    const auto kernel = i8_rows_kernel<MT, XT, ALIGNED, THREADS>;
    const int fit = sgemm_host::blocks_per_sm(regs, dev, kernel, THREADS, smem);
    if (!fit) return SGEMM_ERR_LAUNCH;
    constexpr int warps = THREADS / 32;
    const int blocks = std::min((p.N + warps - 1) / warps, dev.sms * fit);
    return launch(kernel, dim3(blocks), dim3(THREADS), smem, stream, 1, p, X, ldx);
}

template <int MT, int XT, bool ALIGNED>
int rows_by_width(const I8Args &p, const void *X, int64_t ldx, const Device &dev, cudaStream_t stream) {
    const int smem = MT * rows_pitch(p.K);
    return smem > kRowsWide ? launch_rows<MT, XT, ALIGNED, kRowsWideThreads>(p, X, ldx, smem, dev, stream)
                            : launch_rows<MT, XT, ALIGNED, kRowsThreads>(p, X, ldx, smem, dev, stream);
}

// As many tokens at a time as shared memory holds the codes of: all four up to
// K = 57344, two up to 114688, one of any K.  B is read once for each of those.
template <int XT>
int rows_product(const I8Args &all, const void *X, int64_t ldx, const Device &dev, cudaStream_t stream) {
    int most = kRowsTokens;
    while (most * rows_pitch(all.K) > kRowsCodes) most /= 2;
    for (int m = 0; m < all.M; m += most) {
        I8Args p = all;
        p.M = std::min(most, all.M - m);
        p.C = static_cast<char *>(all.C) + m * all.ldc * dtype_size(all.ctype);
        const void *x = X;
        if constexpr (XT < 0) {
            p.A += m * all.lda;
            p.a_scale += m;
        } else {
            x = static_cast<const typename Elem<XT < 0 ? 0 : XT>::type *>(X) + m * ldx;
        }
        auto by_alignment = [&](auto mt) {
            constexpr int MT = decltype(mt)::value;
            return rows16(p.B, p.ldb) ? rows_by_width<MT, XT, true>(p, x, ldx, dev, stream)
                                      : rows_by_width<MT, XT, false>(p, x, ldx, dev, stream);
        };
        const int st = p.M <= 1   ? by_alignment(std::integral_constant<int, 1>{})
                       : p.M <= 2 ? by_alignment(std::integral_constant<int, 2>{})
                                  : by_alignment(std::integral_constant<int, 4>{});
        if (st != SGEMM_OK) return st;
    }
    return SGEMM_OK;
}

// ---------------------------------------------------------------- more tokens

// EARLY: beside the kernel before, which neither reads nor writes these.
template <bool EARLY, class Code>
int lay_out(int rows, int K, const int8_t *q, int64_t ldq, Code *out, int64_t ld, const Device &dev, cudaStream_t stream) {
    const int64_t pieces = (int64_t)rows * ((K + 15) / 16);
    const dim3 grid((unsigned)std::min<int64_t>((pieces + 255) / 256, (int64_t)dev.sms * 8));
    return rows16(q, ldq)
               ? launch<EARLY>(i8_lay_out_kernel<true, Code>, grid, dim3(256), 0, stream, 1, rows, K, q, ldq, out, ld)
               : launch<EARLY>(i8_lay_out_kernel<false, Code>, grid, dim3(256), 0, stream, 1, rows, K, q, ldq, out, ld);
}

int join(const I8Args &p, int splits, const float *partials, int64_t ldp, cudaStream_t stream) {
    const dim3 grid((p.N + 4 * kJoinThreads - 1) / (4 * kJoinThreads), std::min(p.M, 65535));
    return launch(i8_join_kernel, grid, dim3(kJoinThreads), 0, stream, 1, p, splits, partials, ldp);
}

// Tokens a tile, and k-splits: the smallest estimate, in cycles, of rounds over
// the SMs times the length of one, from steps measured on GB300 (208 to 240 tokens
// are taken between 192 and 256), and of adding the splits' sums.  With few
// tokens, few tiles of B: the splits fill the SMs (24 x 16384 x 4096, whose 128
// tiles nearly do, takes 18.5 us whole and 22.6 in two parts); with some hundreds,
// narrower tiles of tokens do, at the price of converting B again for each.
struct StreamPlan {
    int tok = 256, splits = 1;
    StreamPlan() = default;
    StreamPlan(int M, int N, int K, int sms) {
        static constexpr struct {
            int tok, bk;
            double step;
        } kSteps[] = {{16, 128, 760}, {32, 128, 770}, {64, 128, 850}, {128, 128, 1050},
                      {192, 64, 560}, {208, 64, 590}, {224, 64, 620}, {240, 64, 650}, {256, 64, 680}};
        double best = 1e300;
        for (const auto &c : kSteps) {
            const int steps = (K + c.bk - 1) / c.bk;
            const int64_t tiles = (int64_t)((M + c.tok - 1) / c.tok) * ((N + 127) / 128);
            for (int s = 1; s <= 16 && s <= (steps + 3) / 4; ++s) {
                const int64_t rounds = (tiles * s + sms - 1) / sms;
                // a tile's drain shows where there is no second accumulator
                const double drain = c.tok <= 192 ? 1000 : 14. * c.tok;
                double t = (double)rounds * (((steps + s - 1) / s) * c.step + drain) + 2000;
                if (s > 1) t += 5000 + (double)s * M * N * 8 / 1500;
                if (t < best) best = t, tok = c.tok, splits = s;
            }
            if (M <= c.tok) break;
        }
    }
    int64_t ldp(int N) const { return ((int64_t)N + 3) / 4 * 4; }
    int64_t partial_bytes(int M, int N) const { return splits > 1 ? (int64_t)splits * M * ldp(N) * 4 : 0; }
};

template <int TOK>
int launch_stream(const I8Args &p, const __half *x, bool laid_out, const StreamPlan &plan, float *partials,
                  const Device &dev, cudaStream_t stream) {
    using T = I8StreamTile<TOK>;
    static std::atomic<int> regs[sgemm_host::kMaxDevices];
    const auto kernel = i8_stream_kernel<TOK>;
    if (!sgemm_host::blocks_per_sm(regs, dev, kernel, T::THREADS, T::SMEM_BYTES)) return SGEMM_ERR_LAUNCH;
    CUtensorMap tw, tx;
    if (!sgemm_host::encode_i8(&tw, p.B, p.N, p.K, p.ldb, T::ROWS, T::BK) ||
        !sgemm_host::encode_f16(&tx, x, p.M, p.K, ld8(p.K), TOK))
        return SGEMM_ERR_LAUNCH;
    const int64_t units = (int64_t)((p.M + TOK - 1) / TOK) * ((p.N + 127) / 128) * plan.splits;
    return launch<true>(kernel, dim3((unsigned)std::min<int64_t>(units, dev.sms)), dim3(T::THREADS), T::SMEM_BYTES,
                        stream, 1, tw, tx, p, plan.splits, partials, plan.ldp(p.N), (int)laid_out, dev.err_word,
                        sgemm_host::wait_limit_ns(), sgemm_host::test_flags());
}

// The product of FP16 codes x (M x K, on rows of ld8(K)) with the rows of p.B,
// which are first laid out in `rows` where TMA could not read them.
int stream_product(I8Args p, const __half *x, int8_t *rows, float *partials, const StreamPlan &plan, const Device &dev,
                   cudaStream_t stream) {
    int st = SGEMM_OK;
    const bool laid_out = !rows16(p.B, p.ldb);
    if (laid_out) {
        st = lay_out<true>(p.N, p.K, p.B, p.ldb, rows, ld16(p.K), dev, stream);
        if (st != SGEMM_OK) return st;
        p.B = rows;
        p.ldb = ld16(p.K);
    }
    switch (plan.tok) {
        case 16: st = launch_stream<16>(p, x, laid_out, plan, partials, dev, stream); break;
        case 32: st = launch_stream<32>(p, x, laid_out, plan, partials, dev, stream); break;
        case 64: st = launch_stream<64>(p, x, laid_out, plan, partials, dev, stream); break;
        case 128: st = launch_stream<128>(p, x, laid_out, plan, partials, dev, stream); break;
        case 192: st = launch_stream<192>(p, x, laid_out, plan, partials, dev, stream); break;
        case 208: st = launch_stream<208>(p, x, laid_out, plan, partials, dev, stream); break;
        case 224: st = launch_stream<224>(p, x, laid_out, plan, partials, dev, stream); break;
        case 240: st = launch_stream<240>(p, x, laid_out, plan, partials, dev, stream); break;
        default: st = launch_stream<256>(p, x, laid_out, plan, partials, dev, stream);
    }
    if (st != SGEMM_OK || plan.splits == 1) return st;
    return join(p, plan.splits, partials, plan.ldp(p.N), stream);
}

// The workspace of a product: the tokens' scales, their codes as FP16, the rows
// of B where they have to be laid out, and the k-splits' partial sums.
struct Workspace {
    int64_t codes, rows, partials, bytes;
    Workspace(int M, int N, int K, bool lay_out_rows, const StreamPlan &plan) {
        codes = up256(4 * (int64_t)M);
        rows = codes + up256(2 * (int64_t)M * ld8(K));
        partials = rows + (lay_out_rows ? up256((int64_t)N * ld16(K)) : 0);
        bytes = partials + plan.partial_bytes(M, N);
    }
};

int device_sms() {
    Device dev;
    return sgemm_host::device(dev) == SGEMM_OK ? dev.sms : 0;
}

bool output_ok(int M, int N, int K, const signed char *B, int ldb, const float *b_scale, const float *bias,
               const void *C, int ldc, int ctype) {
    if (M < 0 || N < 0 || K < 0 || M > kMaxRows || N > kMaxRows || K > kMaxK || !dtype_ok(ctype)) return false;
    if (ldb < std::max(K, 1) || ldc < std::max(N, 1)) return false;
    if (M == 0 || N == 0) return true;
    if ((K > 0 && !B) || !b_scale || !C || !aligned(b_scale, 4) || !aligned(bias, 4)) return false;
    return aligned(C, (unsigned)dtype_size(ctype));
}

// The output and the workspace against the inputs and each other.  `least` is
// what the workspace has to hold whatever the device; `need` its size, asked
// for last because it queries the device.
template <class Need>
int check_buffers(const Range *in, int n, const Range &c, void *workspace, size_t bytes, size_t least, Need need) {
    for (int i = 0; i < n; ++i)
        if (c.overlaps(in[i])) return SGEMM_ERR_ALIAS;
    const Range ws(bytes ? workspace : nullptr, 1, (int64_t)bytes, (int64_t)bytes, 1);
    if (ws.overlaps(c)) return SGEMM_ERR_ALIAS;
    for (int i = 0; i < n; ++i)
        if (ws.overlaps(in[i])) return SGEMM_ERR_ALIAS;
    if (!aligned(workspace, 16)) return SGEMM_ERR_INVALID_ARG;
    if (least && (!workspace || bytes < least)) return SGEMM_ERR_INVALID_ARG;
    least = need();
    return least && (!workspace || bytes < least) ? SGEMM_ERR_INVALID_ARG : SGEMM_OK;
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
    return quantize(M, K, dtype, x, ldx, reinterpret_cast<int8_t *>(q), ldq, s, dev, stream);
}

// Bytes of a workspace without k-splits, which depend on the device.
static size_t least_workspace(int M, int N, int K, const signed char *B, int ldb) {
    if (M <= 0 || N <= 0 || K <= 0 || takes_rows(M, K)) return 0;
    return (size_t)Workspace(M, N, K, !rows16(reinterpret_cast<const int8_t *>(B), ldb), StreamPlan()).bytes;
}

// One workspace serves both entry points: with 8-bit tokens the place of their
// scales stays unused.
size_t sgemm_i8_workspace_size(int M, int N, int K, const signed char *B, int ldb) {
    if (M <= 0 || N <= 0 || K <= 0 || M > kMaxRows || N > kMaxRows || K > kMaxK || takes_rows(M, K)) return 0;
    const int sms = device_sms();
    if (!sms) return 0;
    return (size_t)Workspace(M, N, K, !rows16(reinterpret_cast<const int8_t *>(B), ldb), StreamPlan(M, N, K, sms)).bytes;
}

int sgemm_i8(int M, int N, int K, const signed char *A, int lda, const float *a_scale, const signed char *B, int ldb,
             const float *b_scale, const float *bias, void *C, int ldc, int ctype, void *workspace,
             size_t workspace_bytes, cudaStream_t stream) {
    if (!output_ok(M, N, K, B, ldb, b_scale, bias, C, ldc, ctype) || lda < std::max(K, 1)) return SGEMM_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return SGEMM_OK;
    if ((K > 0 && !A) || !a_scale || !aligned(a_scale, 4)) return SGEMM_ERR_INVALID_ARG;
    const Range in[5] = {Range(A, M, K, lda, 1), Range(a_scale, 1, M, M, 4), Range(B, N, K, ldb, 1),
                         Range(b_scale, 1, N, N, 4), Range(bias, 1, N, N, 4)};
    int st = check_buffers(in, 5, Range(C, M, N, ldc, dtype_size(ctype)), workspace, workspace_bytes,
                           least_workspace(M, N, K, B, ldb), [&] { return sgemm_i8_workspace_size(M, N, K, B, ldb); });
    if (st != SGEMM_OK) return st;
    Device dev;
    if (sgemm_host::device(dev) != SGEMM_OK) return SGEMM_ERR_DEVICE;
    const I8Args p{M, N, K, reinterpret_cast<const int8_t *>(A), reinterpret_cast<const int8_t *>(B), lda, ldb, a_scale,
                   b_scale, bias, C, ldc, ctype};
    if (K == 0) return join(p, 0, nullptr, 0, stream);
    if (takes_rows(M, K)) return rows_product<-1>(p, nullptr, 0, dev, stream);
    const StreamPlan plan(M, N, K, dev.sms);
    const Workspace at(M, N, K, !rows16(p.B, ldb), plan);
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    __half *codes = reinterpret_cast<__half *>(ws + at.codes);
    st = lay_out<false>(M, K, p.A, lda, codes, ld8(K), dev, stream);
    if (st != SGEMM_OK) return st;
    return stream_product(p, codes, reinterpret_cast<int8_t *>(ws + at.rows), reinterpret_cast<float *>(ws + at.partials),
                          plan, dev, stream);
}

size_t sgemm_linear_i8_workspace_size(int M, int N, int K, const signed char *B, int ldb) {
    return sgemm_i8_workspace_size(M, N, K, B, ldb);
}

int sgemm_linear_i8(int M, int N, int K, int xtype, const void *X, int ldx, const signed char *B, int ldb,
                    const float *b_scale, const float *bias, void *C, int ldc, int ctype, void *workspace,
                    size_t workspace_bytes, cudaStream_t stream) {
    if (!output_ok(M, N, K, B, ldb, b_scale, bias, C, ldc, ctype) || !dtype_ok(xtype) || ldx < std::max(K, 1))
        return SGEMM_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return SGEMM_OK;
    const int size = dtype_size(xtype);
    if (K > 0 && (!X || !aligned(X, (unsigned)size))) return SGEMM_ERR_INVALID_ARG;
    const Range in[4] = {Range(X, M, K, ldx, size), Range(B, N, K, ldb, 1), Range(b_scale, 1, N, N, 4),
                         Range(bias, 1, N, N, 4)};
    int st = check_buffers(in, 4, Range(C, M, N, ldc, dtype_size(ctype)), workspace, workspace_bytes,
                           least_workspace(M, N, K, B, ldb), [&] { return sgemm_linear_i8_workspace_size(M, N, K, B, ldb); });
    if (st != SGEMM_OK) return st;
    Device dev;
    if (sgemm_host::device(dev) != SGEMM_OK) return SGEMM_ERR_DEVICE;
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    float *s = reinterpret_cast<float *>(ws);
    const I8Args p{M, N, K, nullptr, reinterpret_cast<const int8_t *>(B), 0, ldb, s, b_scale, bias, C, ldc, ctype};
    if (K == 0) return join(p, 0, nullptr, 0, stream);
    if (takes_rows(M, K))
        return by_dtype(xtype, [&](auto xt) { return rows_product<decltype(xt)::value>(p, X, ldx, dev, stream); });
    const StreamPlan plan(M, N, K, dev.sms);
    const Workspace at(M, N, K, !rows16(p.B, ldb), plan);
    __half *codes = reinterpret_cast<__half *>(ws + at.codes);
    st = quantize(M, K, xtype, X, ldx, codes, ld8(K), s, dev, stream);
    if (st != SGEMM_OK) return st;
    return stream_product(p, codes, reinterpret_cast<int8_t *>(ws + at.rows), reinterpret_cast<float *>(ws + at.partials),
                          plan, dev, stream);
}

}  // extern "C"
