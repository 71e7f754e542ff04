// The C interface of beam search: argument checks, kernel choice and launch.  The
// contract is in include/sgemm_layers.h.

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "beam.cuh"
#include "host.h"
#include "logprobs_host.h"

namespace {

using namespace sgemm;
using sgemm_host::aligned;
using sgemm_host::Device;
using sgemm_host::dtype_size;
using sgemm_host::launch;
using sgemm_host::Range;

constexpr int kMaxBeams = 32;      // a group's: a warp each
constexpr int kMaxRows = 1 << 30;  // of all groups

bool groups_ok(int B, int W, int top) {
    return B >= 0 && W >= 1 && W <= kMaxBeams && top >= 1 && top <= 32 && (int64_t)B * W <= kMaxRows;
}

// The rows' best logits, their columns, the softmax's references.
struct Workspace {
    int64_t id, reference, bytes;
    Workspace(int64_t T, int top) : id(up256(4 * T * top)), reference(id + up256(4 * T * top)), bytes(reference + up256(8 * T)) {}
    static int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }
};

// The bytes that rows of `outer` runs of `inner` bytes span.
int64_t row_span(int64_t outer, int64_t inner, int64_t run) { return (outer - 1) * run + inner; }

template <int P>
int launch_reorder(ReorderArgs a, int groups, int64_t inner_bytes, const Device &dev, cudaStream_t stream) {
    static std::atomic<int> regs[sgemm_host::kMaxDevices];
    a.inner = inner_bytes / P;
    // two stages of as many rows as there can be parents
    const int smem = 2 * std::min(a.W, a.top) * kReorderThreads * P;
    const int fit = sgemm_host::blocks_per_sm(regs, dev, beam_reorder_kernel<P>, kReorderThreads, smem);
    if (!fit) return SGEMM_ERR_LAUNCH;
    const int64_t blocks = (a.outer * a.inner + kReorderThreads - 1) / kReorderThreads;
    const int y = std::min(groups, 65535);
    const int64_t most = std::max<int64_t>(1, ((int64_t)dev.sms * fit + y - 1) / y);
    for (int g = 0; g < groups; g += 65535) {
        ReorderArgs part = a;
        part.in += (int64_t)g * a.W * a.in_row;
        part.out += (int64_t)g * a.top * a.out_row;
        part.parent += (int64_t)g * a.top;
        const int st = launch(beam_reorder_kernel<P>, dim3((unsigned)std::min(blocks, most), (unsigned)std::min(groups - g, 65535)),
                              dim3(kReorderThreads), (size_t)smem, stream, 1, part);
        if (st != SGEMM_OK) return st;
    }
    return SGEMM_OK;
}

}  // namespace

extern "C" {

size_t sgemm_beam_step_workspace_size(int B, int W, int top) {
    return groups_ok(B, W, top) && B > 0 ? (size_t)Workspace((int64_t)B * W, top).bytes : 0;
}

int sgemm_beam_step(int B, int W, int V, int dtype, const void *logits, int ldz, float scale, const int32_t *mask, int ldm,
                    int mask_rows, const float *score, const unsigned char *finished, int end, int top, float *out_score,
                    int32_t *parent, int32_t *token, void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (!groups_ok(B, W, top)) return SGEMM_ERR_INVALID_ARG;
    const int T = B * W;
    if (!sgemm_host::logprobs_shape_ok(T, V, dtype, sgemm_host::Rows{logits, ldz}, scale, mask, ldm, mask_rows)) return SGEMM_ERR_INVALID_ARG;
    if (finished && end < 0) return SGEMM_ERR_INVALID_ARG;
    if (T == 0) return SGEMM_OK;
    if (!score || !out_score || !parent || !token || !aligned(score, 4) || !aligned(out_score, 4) || !aligned(parent, 4) ||
        !aligned(token, 4))
        return SGEMM_ERR_INVALID_ARG;
    const Workspace at(T, top);
    if (!workspace || !aligned(workspace, 16) || workspace_bytes < (size_t)at.bytes) return SGEMM_ERR_INVALID_ARG;
    const Range in[4] = {Range(logits, T, V, ldz, dtype_size(dtype)), Range(mask, mask_rows, (V + 31) / 32, ldm, 4),
                         Range(score, 1, T, T, 4), Range(finished, 1, T, T, 1)};
    const Range out[4] = {Range(out_score, B, top, top, 4), Range(parent, B, top, top, 4), Range(token, B, top, top, 4),
                          Range(workspace, 1, at.bytes, at.bytes, 1)};
    for (int o = 0; o < 4; ++o) {
        for (const Range &i : in)
            if (out[o].overlaps(i)) return SGEMM_ERR_ALIAS;
        for (int p = 0; p < o; ++p)
            if (out[o].overlaps(out[p])) return SGEMM_ERR_ALIAS;
    }
    Device dev;
    if (sgemm_host::device(dev) != SGEMM_OK) return SGEMM_ERR_DEVICE;
    char *ws = static_cast<char *>(workspace);
    float *value = reinterpret_cast<float *>(ws);
    int32_t *id = reinterpret_cast<int32_t *>(ws + at.id);
    float2 *reference = reinterpret_cast<float2 *>(ws + at.reference);
    const LogprobArgs rows{T, V, logits, ldz, scale, mask, mask_rows > 1 ? ldm : 0, nullptr, nullptr, nullptr, nullptr, top,
                           value, id, score, finished, reference};
    const int st = sgemm_host::by_dtype(dtype, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        return mask ? sgemm_host::logprobs_by_length<DT, true, true>(rows, dev, stream)
                    : sgemm_host::logprobs_by_length<DT, false, true>(rows, dev, stream);
    });
    if (st != SGEMM_OK) return st;
    const BeamArgs a{B, W, top, scale, value, id, reference, score, finished, end, out_score, parent, token};
    return launch<true>(beam_join_kernel, dim3(B), dim3(32 * W), 0, stream, 1, a);
}

int sgemm_beam_reorder(int B, int W, int top, int64_t outer, int64_t inner, const void *in, int64_t in_row, int64_t in_outer,
                       const int32_t *parent, void *out, int64_t out_row, int64_t out_outer, cudaStream_t stream) {
    constexpr int64_t kMost = (int64_t)1 << 44;  // bytes: sums and products of these stay in 64 bits
    if (!groups_ok(B, W, top) || outer < 0 || inner < 0 || outer > kMost || inner > kMost) return SGEMM_ERR_INVALID_ARG;
    if (in_row < 0 || in_outer < 0 || out_row < 0 || out_outer < 0) return SGEMM_ERR_INVALID_ARG;
    if (B == 0 || outer == 0 || inner == 0) return SGEMM_OK;
    if (!in || !out || !parent || !aligned(parent, 4)) return SGEMM_ERR_INVALID_ARG;
    const int64_t rows_in = (int64_t)B * W, rows_out = (int64_t)B * top;
    if (in_row > kMost / rows_in || out_row > kMost / rows_out || in_outer > kMost / outer || out_outer > kMost / outer)
        return SGEMM_ERR_INVALID_ARG;
    // the rows that are written lie apart from each other, whichever of the two levels is the outer one
    const bool apart = (rows_out == 1 || out_row >= row_span(outer, inner, out_outer)) && (outer == 1 || out_outer >= inner);
    const bool within = (outer == 1 || out_outer >= (rows_out - 1) * out_row + inner) && (rows_out == 1 || out_row >= inner);
    if (!apart && !within) return SGEMM_ERR_INVALID_ARG;
    const int64_t bytes_in = (rows_in - 1) * in_row + row_span(outer, inner, in_outer);
    const int64_t bytes_out = (rows_out - 1) * out_row + row_span(outer, inner, out_outer);
    const Range from(in, 1, bytes_in, bytes_in, 1), to(out, 1, bytes_out, bytes_out, 1);
    if (to.overlaps(Range(parent, B, top, top, 4))) return SGEMM_ERR_ALIAS;
    const bool in_place = in == out && in_row == out_row && (outer == 1 || in_outer == out_outer) && top == W;
    if (to.overlaps(from) && !in_place) return SGEMM_ERR_ALIAS;
    Device dev;
    if (sgemm_host::device(dev) != SGEMM_OK) return SGEMM_ERR_DEVICE;
    const ReorderArgs a{W, top, outer, 0, static_cast<const char *>(in), in_row, in_outer, static_cast<char *>(out), out_row,
                        out_outer, parent};
    // the largest pieces that every run consists of and starts on
    uint64_t all = reinterpret_cast<uintptr_t>(in) | reinterpret_cast<uintptr_t>(out) | (uint64_t)inner;
    if (rows_in > 1) all |= (uint64_t)in_row;
    if (rows_out > 1) all |= (uint64_t)out_row;
    if (outer > 1) all |= (uint64_t)in_outer | (uint64_t)out_outer;
    if (all % 16 == 0) return launch_reorder<16>(a, B, inner, dev, stream);
    if (all % 8 == 0) return launch_reorder<8>(a, B, inner, dev, stream);
    if (all % 4 == 0) return launch_reorder<4>(a, B, inner, dev, stream);
    if (all % 2 == 0) return launch_reorder<2>(a, B, inner, dev, stream);
    return launch_reorder<1>(a, B, inner, dev, stream);
}

}  // extern "C"
