// Host-side facts about rows that the row-wise operators share.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "host.h"
#include "row_ring.cuh"

namespace sgemm_host {

using sgemm::row_pieces;

// A matrix of rows as an operator sees it.
struct Rows {
    const void *p;
    int ld;
    // 16-byte pieces: aligned base and rows
    bool vec(int size) const { return !p || (aligned(p, 16) && (int64_t)ld * size % 16 == 0); }
    bool ok(int cols, int size) const { return p && aligned(p, (unsigned)size) && ld >= std::max(cols, 1); }
    Range range(int64_t rows, int cols, int size) const { return Range(p, rows, cols, ld, size); }
    bool same(const Rows &o) const { return p == o.p && ld == o.ld; }
};

// The threads that share a row of D elements, `per` of them each: whole warps.
inline int row_threads(int D, int per) { return ((D + per - 1) / per + 31) / 32 * 32; }

constexpr int kMaxWidth = 24576;  // over a cluster of eight blocks, FP32 rows with every input fit their rings


// How a row is shared out: `ranks` blocks of a cluster with `width` columns
// each, in pieces that no 16 bytes span; `per` elements a thread.  A block
// takes at most `most` threads, and its ring of `slots` rows at most 225 KB.
// Where a warp is enough for a row, a block has four.
struct RowPlan {
    int ranks = 1, width;
    dim3 block;
    size_t smem;
    RowPlan(int D, int size, int slots, int per, int most) : width(D) {
        for (;; ranks *= 2) {
            const int vec = 16 / size;
            width = ranks == 1 ? D : ((D + ranks - 1) / ranks + vec - 1) / vec * vec;
            const int threads = row_threads(width, per);
            block = dim3(threads, threads == 32 && ranks == 1 ? 4 : 1);
            smem = (size_t)slots * row_pieces(threads, per, size) * 16 * block.y;
            if (ranks == 8 || (threads <= most && smem <= 225 * 1024)) break;
        }
    }
    int threads() const { return (int)(block.x * block.y); }
};

// Runners of the gradient's rows: a block (or a cluster of blocks) each, or for
// narrow rows a warp each.  Every one writes its own partial sums, so there are
// no more than the SMs hold at once, 512 threads of 128 registers each; this is
// the most there can be for any type and alignment.
inline int most_grad_runners(int T, int D, int sms) { return std::min(T, std::max(1, 512 * sms / row_threads(D, 16))); }

}  // namespace sgemm_host
