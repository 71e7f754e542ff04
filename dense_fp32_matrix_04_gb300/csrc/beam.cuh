// A step of beam search: of each group's beams the best continuations over the
// vocabulary, and rows of states copied as the beams were chosen.
//
// The rows' best columns and their softmax come from logprobs_kernel, which reads the
// logits once.  What is left is small: W lists of `top` candidates in order, of which
// a candidate's place in the joined list is its place in its own plus, for each other
// list, the number of candidates there that are better, found by halving.
//
// 48 groups of 8 beams over 50001 BF16 logits with 16 continuations take 19.5 us: most of them the pass
// over the logits, 13 instructions a logit beside an occupancy of half the
// SM and three rows an SM where 2.5 would do; 1 group of 4 over 131072 FP32 with a mask 11.6 us,
// launches and a dozen barriers, on 32 of the SMs.  States are copied at the rate of memory: 8 groups of 8 beams,
// 16 x 4001 x 128 BF16 each, 290 us, 6.0 TB/s of the parents read and the rows written; in place,
// where rows that stay are not written, 265.  (Inputs in turn over more than L2 holds.)
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "logprobs.cuh"
#include "ptx.cuh"

namespace sgemm {

struct BeamArgs {
    int B, W, top;
    float scale;
    const float *value;       // T x top: each row's best logits, in order
    const int32_t *id;        // their columns; -1: none
    const float2 *reference;  // T: the largest logit m, and the sum of 2^(z c - fl(m c)), c = scale log2(e)
    const float *score;       // T
    const uint8_t *finished;  // T, or null
    int end;
    float *out_score;         // B x top
    int32_t *parent, *token;
};

// score - ln of the sum relative to the largest's own term: what a candidate's scaled distance from the
// largest is added to.  Of one column, or where no other counts, the quotient is 1 and the score stays as it
// is, so that equal beams which have one way to go on stay equal.  64 bits where FP32 would round numbers
// of the size of the score (the fraction has a logarithm below 0.7, which FP32 has to 2^-25).
__device__ __forceinline__ double beam_base(float score, float2 r, float scale) {
    const float c = scale * kLog2e, M = SoftmaxState::reference(r.x, c);
    const float own = SoftmaxState::usual(M) ? exp2_approx(fmaf(r.x, c, -M)) : 1.f;  // as the pass computes it
    const uint32_t bits = __float_as_uint(__fdiv_rn(r.y, own));
    const int e = (int)(bits >> 23) - 127;
    const float f = __uint_as_float((bits & 0x7fffffu) | 0x3f800000u);
    return (double)score - fma((double)e, 0.6931471805599453, (double)logf(f));
}

// A whole number in the order of the values (not NaN): comparisons in 64 bits without the few units
// that there are for FP64.
__device__ __forceinline__ int64_t ordered(double v) {
    const int64_t b = __double_as_longlong(v + 0.0);  // (of the two zeros the positive one)
    return b >= 0 ? b : b ^ 0x7fffffffffffffffll;
}

// A block a group, a warp a beam.
__global__ void __launch_bounds__(1024) beam_join_kernel(const BeamArgs a) {
    __shared__ int64_t list[32][32];
    __shared__ double base[32], largest[32];
    const int beam = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row0 = (int64_t)blockIdx.x * a.W;
    griddep_wait();
    // a lane of the first warp a beam: FP64 takes a warp as long for one lane as for all
    if (beam == 0 && lane < a.W) {
        const float score = a.score[row0 + lane];
        const bool goes_on = row_takes_part(score, a.finished ? a.finished + row0 + lane : nullptr);
        const float2 r = goes_on ? a.reference[row0 + lane] : make_float2(0.f, 1.f);
        base[lane] = goes_on ? beam_base(score, r, a.scale) : (double)score;
        largest[lane] = (double)r.x;
    }
    const int64_t row = row0 + beam;
    const float score = a.score[row];
    const bool ended = a.finished && a.finished[row];
    int token = -1;
    float z = 0.f;
    if (lane < a.top && row_takes_part(score, nullptr)) {
        if (ended) {
            if (lane == 0) token = a.end;
        } else {
            token = a.id[row * a.top + lane];
            z = a.value[row * a.top + lane];
        }
    }
    __syncthreads();
    // candidates of different beams may lie closer than FP32 tells apart
    const double v = token < 0 ? -INFINITY : fma((double)z - largest[beam], (double)a.scale, base[beam]);
    const int64_t key = ordered(v);
    list[beam][lane] = key;
    __syncthreads();
    if (lane >= a.top) return;
    int place = lane;
    for (int j = 0; j < a.W; ++j) {
        if (j == beam) continue;
        // the candidates of beam j that come first: the larger ones, and of a lower beam the equal ones
        const int64_t least = j < beam ? key : key + 1;
        int n = 0;
#pragma unroll
        for (int step = 32; step; step >>= 1)
            if (n + step <= a.top && list[j][n + step - 1] >= least) n += step;
        place += n;
    }
    if (place >= a.top) return;
    const int64_t at = (int64_t)blockIdx.x * a.top + place;
    const bool has = v > -INFINITY;
    a.out_score[at] = (float)v;
    a.parent[at] = has ? beam : -1;
    a.token[at] = has ? token : -1;
}

// ---------------------------------------------------------------- reordering

struct ReorderArgs {
    int W, top;
    int64_t outer, inner;  // a row: `outer` runs of `inner` pieces
    const char *in;
    int64_t in_row, in_outer;    // bytes between rows, and between runs
    char *out;
    int64_t out_row, out_outer;
    const int32_t *parent;       // B x top
};

// A piece of P bytes to shared memory, asynchronously where the size allows it.
template <int P>
__device__ __forceinline__ void copy_piece(char *to, const char *from) {
    if constexpr (P == 16) {
        cp_async_16(smem_addr(to), from, 16);
    } else if constexpr (P == 8) {
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;\n" ::"r"(smem_addr(to)), "l"(from) : "memory");
    } else if constexpr (P == 4) {
        cp_async_4(smem_addr(to), from, 4);
    } else if constexpr (P == 2) {
        *reinterpret_cast<uint16_t *>(to) = *reinterpret_cast<const uint16_t *>(from);
    } else {
        *to = *from;
    }
}
template <int P>
struct PieceType;
template <> struct PieceType<16> { using type = uint4; };
template <> struct PieceType<8> { using type = uint2; };
template <> struct PieceType<4> { using type = uint32_t; };
template <> struct PieceType<2> { using type = uint16_t; };
template <> struct PieceType<1> { using type = uint8_t; };

// blockIdx.y: a group.  A thread takes one piece of each of the group's rows that a
// beam is copied from into its own places of shared memory, and only then writes the
// rows that change, so states may be reordered in place; each parent is read once.
// The next pieces are on their way while these are written.
constexpr int kReorderThreads = 128;
template <int P>
__global__ void __launch_bounds__(kReorderThreads) beam_reorder_kernel(const ReorderArgs a) {
    using type = typename PieceType<P>::type;
    extern __shared__ __align__(16) char pieces[];  // 2 stages x rows that are read x threads
    __shared__ int source[32], to_row[32], to_place[32], counts[2];
    const int64_t group = blockIdx.y;
    if (threadIdx.x < 32) {
        // rows that are written (child and its parent), and the parents among them
        const int child = threadIdx.x;
        int p = child < a.top ? a.parent[group * a.top + child] : -1;
        if (p < 0 || p >= a.W || (a.in == a.out && p == child)) p = -1;
        uint32_t needed = p >= 0 ? 1u << p : 0u;
        needed = __reduce_or_sync(0xffffffffu, needed);
        const uint32_t written = __ballot_sync(0xffffffffu, p >= 0);
        const int place = p >= 0 ? __popc(needed & ((1u << p) - 1)) : 0;
        if (p >= 0) {
            const int at = __popc(written & ((1u << child) - 1));
            to_row[at] = child;
            to_place[at] = place;
        }
        if (needed >> child & 1) source[__popc(needed & ((1u << child) - 1))] = child;
        if (child == 0) counts[0] = __popc(needed), counts[1] = __popc(written);
    }
    __syncthreads();
    const int n_read = counts[0], n_write = counts[1];
    if (!n_write) return;
    const char *in = a.in + group * a.W * a.in_row;
    char *out = a.out + group * a.top * a.out_row;
    const int64_t step = (int64_t)gridDim.x * kReorderThreads, step_o = step / a.inner, step_i = step % a.inner;
    // this thread's next piece to copy: run o, place i in it
    struct At {
        int64_t o, i;
    };
    auto advance = [&](At &p) {
        p.o += step_o;
        p.i += step_i;
        if (p.i >= a.inner) p.i -= a.inner, ++p.o;
    };
    const int64_t first = (int64_t)blockIdx.x * kReorderThreads + threadIdx.x;
    At ahead{first / a.inner, first % a.inner}, now = ahead;
    char *mine = pieces + threadIdx.x * P;
    auto fetch = [&](int stage) {
        if (ahead.o < a.outer) {
            const char *from = in + ahead.o * a.in_outer + ahead.i * P;
            for (int r = 0; r < n_read; ++r)
                copy_piece<P>(mine + (stage * n_read + r) * kReorderThreads * P, from + source[r] * a.in_row);
        }
        cp_async_commit();
        advance(ahead);
    };
    fetch(0);
    for (int stage = 0; now.o < a.outer; stage ^= 1) {
        fetch(stage ^ 1);
        cp_async_wait<1>();
        char *to = out + now.o * a.out_outer + now.i * P;
        for (int k = 0; k < n_write; ++k)
            *reinterpret_cast<type *>(to + to_row[k] * a.out_row) =
                *reinterpret_cast<const type *>(mine + (stage * n_read + to_place[k]) * kReorderThreads * P);
        advance(now);
    }
}

}  // namespace sgemm
