// The C interface of the products with 4-bit weights: argument checks, kernel
// choice and launch.  The contract is in include/sgemm_layers.h.

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/sgemm_layers_testing.h"
#include "fp4_mma.cuh"
#include "fp4_pair.cuh"
#include "fp4_quantize.cuh"
#include "fp4_rows.cuh"
#include "host.h"

namespace {

using namespace sgemm;
using sgemm_host::aligned;
using sgemm_host::by_dtype;
using sgemm_host::Device;
using sgemm_host::dtype_ok;
using sgemm_host::dtype_size;
using sgemm_host::launch;
using sgemm_host::Range;

constexpr int kMaxRows = 1 << 30;     // row numbers and a round of them fit 32 bits
constexpr int kMaxColumns = 1 << 24;  // a tile's products over more would come near the limit of a wait

bool block_ok(int block) { return block == 16 || block == 32; }
int64_t code_bytes(int K) { return ((int64_t)K + 1) / 2; }
int64_t code_pitch(int K) { return (code_bytes(K) + 15) / 16 * 16; }
int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }
int64_t tile_bytes(int rows, int K, int block) {
    return rows > 0 && K > 0 ? ((int64_t)rows + 127) / 128 * fp4_tiles(K, block) * kFp4TileBytes : 0;
}

// Calls f(std::integral_constant<int, block>).
template <class F>
int by_block(int block, F &&f) {
    return block == 16 ? f(std::integral_constant<int, 16>{}) : f(std::integral_constant<int, 32>{});
}

// ---------------------------------------------------------------- quantising

template <int DT, bool ALIGNED, int BLOCK, int EACH>
int launch_quantize_rows(const Fp4Rows &a, const void *x, int64_t ldx, const Device &dev, cudaStream_t stream) {
    using type = typename Elem<DT>::type;
    static std::atomic<int> regs[sgemm_host::kMaxDevices];
    const auto kernel = quantize_fp4_kernel<DT, ALIGNED, BLOCK, EACH>;
    const int threads = (a.K + 512 * EACH - 1) / (512 * EACH) * 32;
    const dim3 block(threads, threads == 32 ? 4 : 1);
    const int smem = kFp4RowSlots * EACH * Fp4Piece<DT, ALIGNED>::WARP_PIECES * 16 * (int)(block.x * block.y / 32);
    const int fit = sgemm_host::blocks_per_sm(regs, dev, kernel, (int)(block.x * block.y), smem);
    if (!fit) return SGEMM_ERR_LAUNCH;
    const int64_t groups = ((int64_t)a.rows + block.y - 1) / block.y;
    return launch(kernel, dim3((unsigned)std::min<int64_t>(groups, (int64_t)dev.sms * fit)), block, (size_t)smem, stream, 1, a,
                  static_cast<const type *>(x), ldx);
}

template <int DT, bool ALIGNED, int BLOCK>
int launch_quantize(const Fp4Rows &a, const void *x, int64_t ldx, const Device &dev, cudaStream_t stream) {
    using type = typename Elem<DT>::type;
    if (a.K > 16384) {
        static std::atomic<int> regs[sgemm_host::kMaxDevices];
        const auto kernel = quantize_fp4_wide_kernel<DT, ALIGNED, BLOCK>;
        const int fit = sgemm_host::blocks_per_sm(regs, dev, kernel, 1024, 0);
        if (!fit) return SGEMM_ERR_LAUNCH;
        return launch(kernel, dim3((unsigned)std::min(a.rows, dev.sms * fit)), dim3(1024), 0, stream, 1, a,
                      static_cast<const type *>(x), ldx);
    }
    return a.K <= 4096 ? launch_quantize_rows<DT, ALIGNED, BLOCK, 1>(a, x, ldx, dev, stream)
                       : launch_quantize_rows<DT, ALIGNED, BLOCK, 2>(a, x, ldx, dev, stream);
}

int quantize(const Fp4Rows &a, int dtype, int block, const void *x, int64_t ldx, const Device &dev, cudaStream_t stream) {
    return by_dtype(dtype, [&](auto dt) {
        constexpr int DT = decltype(dt)::value, VEC = Elem<DT>::VEC;
        const bool vec = a.K % VEC == 0 && aligned(x, 16) && ldx % VEC == 0;
        return by_block(block, [&](auto b) {
            constexpr int BLOCK = decltype(b)::value;
            return vec ? launch_quantize<DT, true, BLOCK>(a, x, ldx, dev, stream)
                       : launch_quantize<DT, false, BLOCK>(a, x, ldx, dev, stream);
        });
    });
}

// ---------------------------------------------------------------- the product

// How a product is shared out: tiles of 16 to 128 tokens on one SM, for which the
// blocks of a cluster can split K, or of 256 on a pair.  The smallest estimate, in
// cycles, of rounds over the SMs times the length of one, from times on GB300 (a step
// is 256 columns; a round is no shorter than what it stores takes).  A split costs a
// cluster's launch, two of its barriers and the join: worth it for long rows only
// (weights in turn: 16 x 4096 x 16384 18.4 us whole, 12.2 in four parts; x 4096 7.8 and 7.5;
// 64 x 4096 x 4096 8.2 and 9.4).  Pairs take a cluster's launch too: on single SMs and on pairs
// 600 x 4096 x 4096 takes 13.4 and 11.8 us, 512 tokens 9.1 and 11.7, 2432 x 4096 x 1024 11.7
// and 13.2, 8192 x 8192 x 1024 55 and 42.
struct Fp4Plan {
    int tok = 16, splits = 1;  // tok 256: a pair
    Fp4Plan(int M, int N, int K, int sms) {
        static constexpr struct {
            int tok;
            double step, round, least;
        } kSteps[] = {{16, 395, 600, 0}, {32, 395, 600, 0}, {64, 400, 800, 2400}, {128, 450, 1200, 3100}, {256, 610, 1300, 5000}};
        double best = 1e300;
        const int steps = (K + 255) / 256;
        for (const auto &c : kSteps) {
            if (c.tok < 64 && M > c.tok) continue;  // see Fp4Tile
            const bool pair = c.tok == 256;
            const int64_t tiles = (int64_t)((M + c.tok - 1) / c.tok) * ((N + (pair ? 255 : 127)) / (pair ? 256 : 128));
            const int slots = pair ? sms / 2 : sms;
            // (clusters of four leave some SMs without a block)
            for (int s = 1; s == 1 || (!pair && s <= 4 && s <= steps && tiles * s <= sms - 8); s *= 2) {
                const int64_t rounds = (tiles * s + slots - 1) / slots;
                double t = (double)rounds * std::max(((steps + s - 1) / s) * c.step + c.round, c.least);
                if (s > 1) t += 1300 + 112. * c.tok;
                if (pair) t += 3500;
                if (t < best) best = t, tok = c.tok, splits = s;
            }
            if (M <= c.tok) break;
        }
    }
};

struct Fp4Operands {
    const uint8_t *A, *B;
    int64_t lda, ldb;
};

// launch, beside the kernel before where `early` holds.
template <class... Params, class... Args>
int launch_beside(bool early, void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, unsigned cluster,
                  Args &&...args) {
    return early ? launch<true>(kernel, grid, block, smem, stream, cluster, std::forward<Args>(args)...)
                 : launch(kernel, grid, block, smem, stream, cluster, std::forward<Args>(args)...);
}

template <int TOK, int BLOCK>
int launch_mma(const Fp4Args &p, const Fp4Operands &o, int splits, bool early, const Device &dev, cudaStream_t stream) {
    using T = Fp4Tile<TOK, BLOCK>;
    static std::atomic<int> regs[sgemm_host::kMaxDevices];
    const auto kernel = fp4_mma_kernel<TOK, BLOCK>;
    if (!sgemm_host::blocks_per_sm(regs, dev, kernel, T::THREADS, T::SMEM_BYTES)) return SGEMM_ERR_LAUNCH;
    CUtensorMap tw, tx;
    if (!sgemm_host::encode_i8(&tw, o.B, p.N, code_bytes(p.K), o.ldb, T::ROWS, T::BYTES) ||
        !sgemm_host::encode_i8(&tx, o.A, p.M, code_bytes(p.K), o.lda, TOK, T::BYTES))
        return SGEMM_ERR_LAUNCH;
    const int64_t units = (int64_t)((p.M + TOK - 1) / TOK) * ((p.N + T::ROWS - 1) / T::ROWS) * splits;
    return launch_beside(early, kernel, dim3((unsigned)(splits > 1 ? units : std::min<int64_t>(units, dev.sms))), dim3(T::THREADS),
                         T::SMEM_BYTES, stream, (unsigned)splits, tw, tx, p, splits, dev.err_word, sgemm_host::wait_limit_ns(),
                         sgemm_host::test_flags());
}

template <int BLOCK>
int launch_pair(const Fp4Args &p, const Fp4Operands &o, bool early, const Device &dev, cudaStream_t stream) {
    using T = Fp4PairTile<BLOCK>;
    static std::atomic<int> regs[sgemm_host::kMaxDevices];
    const auto kernel = fp4_pair_kernel<BLOCK>;
    if (!sgemm_host::blocks_per_sm(regs, dev, kernel, T::THREADS, T::SMEM_BYTES)) return SGEMM_ERR_LAUNCH;
    const int64_t words = (int64_t)fp4_tiles(p.K, BLOCK) * (kFp4TileBytes / 8);
    CUtensorMap tw, tx, tws, txs;
    if (!sgemm_host::encode_i8(&tw, o.B, p.N, code_bytes(p.K), o.ldb, T::ROWS / 2, T::BYTES) ||
        !sgemm_host::encode_i8(&tx, o.A, p.M, code_bytes(p.K), o.lda, T::TOK / 2, T::BYTES) ||
        !sgemm_host::encode_words(&tws, p.b_tiles, (p.N + 127) / 128, words, 1, T::WS_BYTES / 8) ||
        !sgemm_host::encode_words(&txs, p.a_tiles, (p.M + 127) / 128, words, 2, T::WS_BYTES / 8))
        return SGEMM_ERR_LAUNCH;
    const int64_t tiles = (int64_t)((p.M + T::TOK - 1) / T::TOK) * ((p.N + T::ROWS - 1) / T::ROWS);
    return launch_beside(early, kernel, dim3((unsigned)(2 * std::min<int64_t>(tiles, dev.sms / 2))), dim3(T::THREADS), T::SMEM_BYTES,
                         stream, 2, tw, tx, tws, txs, p, dev.err_word, sgemm_host::wait_limit_ns(), sgemm_host::test_flags());
}

// One token whose codes fit shared memory goes to the kernel that reads whole rows (by 4096 x 4096,
// weights in turn, 5.7 us there, on the tensor cores 7.5).
bool takes_rows(int M, int K) { return M == 1 && fp4_rows_smem(K) <= kFp4RowsSmem; }

template <int XT, int BLOCK>
int launch_rows(const Fp4RowsArgs &a, const Device &dev, cudaStream_t stream) {
    static std::atomic<int> regs[sgemm_host::kMaxDevices];
    const auto kernel = fp4_rows_kernel<XT, BLOCK>;
    const int smem = (int)fp4_rows_smem(a.p.K);
    const int fit = sgemm_host::blocks_per_sm(regs, dev, kernel, kFp4RowsThreads, smem);
    if (!fit) return SGEMM_ERR_LAUNCH;
    const int groups = (a.p.N + 127) / 128 * 8;
    return launch(kernel, dim3((unsigned)std::min(groups, dev.sms * fit)), dim3(kFp4RowsThreads), (size_t)smem, stream, 1, a);
}

// xtype -1: the token is codes.
int rows_product(const Fp4RowsArgs &a, int xtype, int block, const Device &dev, cudaStream_t stream) {
    return by_block(block, [&](auto b) {
        constexpr int BLOCK = decltype(b)::value;
        if (xtype < 0) return launch_rows<-1, BLOCK>(a, dev, stream);
        return by_dtype(xtype, [&](auto xt) { return launch_rows<decltype(xt)::value, BLOCK>(a, dev, stream); });
    });
}

// early: the kernel before is this call's own, which does not write B.
int product(const Fp4Args &p, const Fp4Operands &o, int block, bool early, const Device &dev, cudaStream_t stream) {
    const Fp4Plan plan(p.M, p.N, p.K, dev.sms);
    return by_block(block, [&](auto b) {
        constexpr int BLOCK = decltype(b)::value;
        switch (plan.tok) {
            case 16: return launch_mma<16, BLOCK>(p, o, plan.splits, early, dev, stream);
            case 32: return launch_mma<32, BLOCK>(p, o, plan.splits, early, dev, stream);
            case 64: return launch_mma<64, BLOCK>(p, o, plan.splits, early, dev, stream);
            case 128: return launch_mma<128, BLOCK>(p, o, plan.splits, early, dev, stream);
            default: return launch_pair<BLOCK>(p, o, early, dev, stream);
        }
    });
}

int empty_product(const Fp4Args &p, const Device &dev, cudaStream_t stream) {
    const int64_t blocks = ((int64_t)p.M * p.N + 255) / 256;
    return launch(fp4_empty_kernel, dim3((unsigned)std::min<int64_t>(blocks, dev.sms * 8)), dim3(256), 0, stream, 1, p);
}

// Rows of codes, which start on 16 bytes, with their scales.
bool codes_ok(const unsigned char *q, int ld, const unsigned char *tiles, const float *scale, int K) {
    if (K > 0 && (!q || !tiles || !aligned(q, 16) || ld % 16 != 0 || !aligned(tiles, 16))) return false;
    return aligned(scale, 4);
}

bool shapes_ok(int M, int N, int K, int block, int ldb, int ldc, int ctype) {
    if (M < 0 || N < 0 || K < 0 || M > kMaxRows || N > kMaxRows || K > kMaxColumns) return false;
    return block_ok(block) && dtype_ok(ctype) && ldb >= std::max<int64_t>(code_bytes(K), 1) && ldc >= std::max(N, 1);
}

bool output_ok(const void *C, int ctype, const float *bias) {
    return C && aligned(C, (unsigned)dtype_size(ctype)) && aligned(bias, 4);
}

}  // namespace

extern "C" {

int sgemm_fp4_plan_model(int M, int N, int K, int sms, int *tokens, int *parts) {
    if (!tokens || !parts || M < 1 || N < 1 || K < 1 || M > kMaxRows || N > kMaxRows || K > kMaxColumns || sms < 2)
        return SGEMM_ERR_INVALID_ARG;
    const Fp4Plan plan(M, N, K, sms);
    const bool rows = takes_rows(M, K);
    *tokens = rows ? 1 : plan.tok;
    *parts = rows ? 1 : plan.splits;
    return SGEMM_OK;
}

size_t sgemm_fp4_scales_size(int rows, int K, int block) {
    if (rows < 0 || K < 0 || rows > kMaxRows || K > kMaxColumns || !block_ok(block)) return 0;
    return (size_t)tile_bytes(rows, K, block);
}

int sgemm_quantize_fp4(int M, int K, int dtype, const void *x, int ldx, int block, unsigned char *q, int ldq,
                       unsigned char *block_scale, float *scale, cudaStream_t stream) {
    if (M < 0 || K < 0 || M > kMaxRows || K > kMaxColumns || !dtype_ok(dtype) || !block_ok(block)) return SGEMM_ERR_INVALID_ARG;
    if (ldx < std::max(K, 1) || ldq < std::max<int64_t>(code_bytes(K), 1)) return SGEMM_ERR_INVALID_ARG;
    if ((block == 16) != (scale != nullptr) && M > 0) return SGEMM_ERR_INVALID_ARG;
    if (M == 0) return SGEMM_OK;
    const int size = dtype_size(dtype);
    if (!aligned(scale, 4)) return SGEMM_ERR_INVALID_ARG;
    if (K > 0 && (!x || !aligned(x, (unsigned)size) || !codes_ok(q, ldq, block_scale, nullptr, K))) return SGEMM_ERR_INVALID_ARG;
    const int64_t n = tile_bytes(M, K, block);
    const Range in(x, M, K, ldx, size);
    const Range out[3] = {Range(q, M, code_bytes(K), ldq, 1), Range(block_scale, 1, n, n, 1), Range(scale, 1, M, M, 4)};
    for (int o = 0; o < 3; ++o) {
        if (out[o].overlaps(in)) return SGEMM_ERR_ALIAS;
        for (int i = 0; i < o; ++i)
            if (out[o].overlaps(out[i])) return SGEMM_ERR_ALIAS;
    }
    if (K == 0) {
        if (scale && cudaMemsetAsync(scale, 0, (size_t)M * sizeof(float), stream) != cudaSuccess) {
            (void)cudaGetLastError();
            return SGEMM_ERR_LAUNCH;
        }
        return SGEMM_OK;
    }
    Device dev;
    if (sgemm_host::device(dev) != SGEMM_OK) return SGEMM_ERR_DEVICE;
    return quantize({M, (M + 127) / 128 * 128, K, q, ldq, block_scale, scale}, dtype, block, x, ldx, dev, stream);
}

int sgemm_fp4_lay_out_scales(int rows, int K, int block, const unsigned char *s, int lds, unsigned char *tiles,
                             cudaStream_t stream) {
    if (rows < 0 || K < 0 || rows > kMaxRows || K > kMaxColumns || !block_ok(block)) return SGEMM_ERR_INVALID_ARG;
    if (rows == 0 || K == 0) return SGEMM_OK;
    const int blocks = fp4_blocks(K, block);
    if (!s || lds < blocks || !tiles || !aligned(tiles, 16)) return SGEMM_ERR_INVALID_ARG;
    const int64_t n = tile_bytes(rows, K, block);
    if (Range(tiles, 1, n, n, 1).overlaps(Range(s, rows, blocks, lds, 1))) return SGEMM_ERR_ALIAS;
    Device dev;
    if (sgemm_host::device(dev) != SGEMM_OK) return SGEMM_ERR_DEVICE;
    const int64_t most = (n / 4 + 255) / 256;
    return launch(fp4_lay_out_scales_kernel, dim3((unsigned)std::min<int64_t>(most, dev.sms * 8)), dim3(256), 0, stream, 1,
                  rows, blocks, s, (int64_t)lds, tiles);
}

int sgemm_fp4(int M, int N, int K, int block, const unsigned char *A, int lda, const unsigned char *a_block,
              const float *a_scale, const unsigned char *B, int ldb, const unsigned char *b_block, const float *b_scale,
              const float *bias, void *C, int ldc, int ctype, cudaStream_t stream) {
    if (!shapes_ok(M, N, K, block, ldb, ldc, ctype) || lda < std::max<int64_t>(code_bytes(K), 1)) return SGEMM_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return SGEMM_OK;
    if (!output_ok(C, ctype, bias) || !codes_ok(A, lda, a_block, a_scale, K) || !codes_ok(B, ldb, b_block, b_scale, K))
        return SGEMM_ERR_INVALID_ARG;
    const int64_t na = tile_bytes(M, K, block), nb = tile_bytes(N, K, block);
    const Range c(C, M, N, ldc, dtype_size(ctype));
    for (const Range &in : {Range(A, M, code_bytes(K), lda, 1), Range(a_block, 1, na, na, 1), Range(a_scale, 1, M, M, 4),
                            Range(B, N, code_bytes(K), ldb, 1), Range(b_block, 1, nb, nb, 1), Range(b_scale, 1, N, N, 4),
                            Range(bias, 1, N, N, 4)})
        if (c.overlaps(in)) return SGEMM_ERR_ALIAS;
    Device dev;
    if (sgemm_host::device(dev) != SGEMM_OK) return SGEMM_ERR_DEVICE;
    const Fp4Args p{M, N, K, a_block, b_block, a_scale, b_scale, bias, C, ldc, ctype};
    if (K == 0) return empty_product(p, dev, stream);
    if (takes_rows(M, K)) return rows_product({p, A, B, ldb, nullptr}, -1, block, dev, stream);
    return product(p, {A, B, lda, ldb}, block, false, dev, stream);
}

// The tokens' codes, their block scales, their scales.
size_t sgemm_linear_fp4_workspace_size(int M, int K, int block) {
    if (M <= 0 || K <= 0 || M > kMaxRows || K > kMaxColumns || !block_ok(block) || takes_rows(M, K)) return 0;
    return (size_t)(up256((int64_t)M * code_pitch(K)) + up256(tile_bytes(M, K, block)) + (block == 16 ? up256((int64_t)M * 4) : 0));
}

int sgemm_linear_fp4(int M, int N, int K, int xtype, const void *X, int ldx, int block, const unsigned char *B, int ldb,
                     const unsigned char *b_block, const float *b_scale, const float *bias, void *C, int ldc, int ctype,
                     void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (!shapes_ok(M, N, K, block, ldb, ldc, ctype) || !dtype_ok(xtype) || ldx < std::max(K, 1)) return SGEMM_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return SGEMM_OK;
    const int size = dtype_size(xtype);
    if (!output_ok(C, ctype, bias) || !codes_ok(B, ldb, b_block, b_scale, K) || (K > 0 && (!X || !aligned(X, (unsigned)size))))
        return SGEMM_ERR_INVALID_ARG;
    const size_t need = sgemm_linear_fp4_workspace_size(M, K, block);
    if (!aligned(workspace, 16) || (need && (!workspace || workspace_bytes < need))) return SGEMM_ERR_INVALID_ARG;
    const int64_t nb = tile_bytes(N, K, block);
    const Range c(C, M, N, ldc, dtype_size(ctype)), ws(need ? workspace : nullptr, 1, (int64_t)need, (int64_t)need, 1);
    for (const Range &in : {Range(X, M, K, ldx, size), Range(B, N, code_bytes(K), ldb, 1), Range(b_block, 1, nb, nb, 1),
                            Range(b_scale, 1, N, N, 4), Range(bias, 1, N, N, 4)})
        if (c.overlaps(in) || ws.overlaps(in)) return SGEMM_ERR_ALIAS;
    if (c.overlaps(ws)) return SGEMM_ERR_ALIAS;
    Device dev;
    if (sgemm_host::device(dev) != SGEMM_OK) return SGEMM_ERR_DEVICE;
    Fp4Args p{M, N, K, nullptr, b_block, nullptr, b_scale, bias, C, ldc, ctype};
    if (K == 0) return empty_product(p, dev, stream);
    if (takes_rows(M, K)) return rows_product({p, nullptr, B, ldb, X}, xtype, block, dev, stream);
    uint8_t *codes = static_cast<uint8_t *>(workspace), *tiles = codes + up256((int64_t)M * code_pitch(K));
    float *scale = block == 16 ? reinterpret_cast<float *>(tiles + up256(tile_bytes(M, K, block))) : nullptr;
    const int st = quantize({M, M, K, codes, code_pitch(K), tiles, scale}, xtype, block, X, ldx, dev, stream);
    if (st != SGEMM_OK) return st;
    p.a_tiles = tiles;
    p.a_scale = scale;
    return product(p, {codes, B, code_pitch(K), ldb}, block, true, dev, stream);
}

}  // extern "C"
