// Log probabilities of given columns, entropy, log-sum-exp and the most likely
// columns of rows of logits, in one pass over them; and the gradient.
//
// With m the largest logit seen, c = scale log2(e), M = m c rounded to FP32 and
// t_j = z_j c - M (one fused operation), the pass keeps
//     s = sum 2^t_j   and   s1 = sum 2^t_j t_j,
// which a larger M' turns into f s and f (s1 + s d), d = M - M', f = 2^d: the
// rounding of M is the same for every term, so it costs no accuracy while it is
// below 1/2 (|M| < 2^24; the 2^128 that FP32 ends at is one of 128).  At the end
// lse = ln 2 M + ln s, taken as scale m + ln s + ln 2 (M - m c) with an exact
// difference; entropy = ln s - ln 2 s1 / s; log p_y = scale (z_y - m) - ln s -
// ln 2 (M - m c).  Where m c is larger (rows of nothing but mask values, large
// scales), t_j = (z_j - m) c instead.
//
// The alternatives cost the pass no instruction a column: each thread knows the
// largest logit it has met, and at the row's end at least `top` columns reach the
// top-th largest of the maxima of 32 groups of threads.  Only the threads that
// have such a column, a handful, have theirs looked at again, and the few columns
// that reach it are ranked against each other.  That is a dozen barriers and a
// second look at a part of the row, which grows with top and V: 4096 x 50001 takes
// 80 us without alternatives and 89 with five, 4096 x 100001 205 with twenty.
//
// Of 16-bit logits the pass is bound by the issue of instructions (about 12 an
// element, one of them the exponential, which alone would take 44 us at 4096 x
// 50001): 89 us there, 4.6 TB/s, against 60.5 for the bytes.  A masked column is
// -infinity, whose term 0 times -infinity is NaN, so a chunk with one is added a
// second time, column by column: 4096 x 50001 takes 181 us with a mask, FP32 4096
// x 32000 115 against 92.  Three rows of 131072 with 20 alternatives, shared by 24
// blocks, take 13 us: a latency to read, one to join a cluster, and the row's end.
// The gradient reads and writes once: 4096 x 32000 FP32 151 us, 511 x 128001 BF16
// 50 us (5.2 TB/s).
#pragma once

#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "ptx.cuh"
#include "rows.cuh"

namespace sgemm {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct LogprobArgs {
    int T, V;
    const void *z;
    int64_t ldz;
    float scale;
    const int32_t *mask;
    int64_t ldm;       // words between the mask's rows; 0: one row for all
    const int64_t *target;
    float *logprob, *entropy, *lse;
    int top;
    float *top_logprob;
    int32_t *top_id;
};

__device__ __forceinline__ float exp2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(x));
    return r;
}

// The same with results below 2^-126, which exp2_approx takes as 0.
__device__ __forceinline__ float exp2_small(float x) {
    float r;
    asm("ex2.approx.f32 %0, %1;\n" : "=f"(r) : "f"(x));
    return r;
}

// Bits of the mask's row for columns c .. c + n - 1 (n <= 8), lowest first;
// columns from V on read as 0.
__device__ __forceinline__ uint32_t mask_bits(const int32_t *row, int c, int n, int V) {
    const int w = c >> 5, s = c & 31;
    uint32_t lo = (uint32_t)row[w], hi = 0;
    if (s + n > 32 && (w + 1) * 32 < V) hi = (uint32_t)row[w + 1];
    return __funnelshift_r(lo, hi, s);
}

// The largest of the 16 bytes' elements (a NaN only where all are).
template <int DT>
__device__ __forceinline__ float max16(const uint4 &raw) {
    if constexpr (DT == SGEMM_F32) {
        return fmaxf(fmaxf(__uint_as_float(raw.x), __uint_as_float(raw.y)),
                     fmaxf(__uint_as_float(raw.z), __uint_as_float(raw.w)));
    } else if constexpr (DT == SGEMM_BF16) {
        auto h = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162 *>(&w); };
        const __nv_bfloat162 m = __hmax2(__hmax2(h(raw.x), h(raw.y)), __hmax2(h(raw.z), h(raw.w)));
        return fmaxf(__low2float(m), __high2float(m));
    } else {
        auto h = [](uint32_t w) { return *reinterpret_cast<const __half2 *>(&w); };
        const __half2 m = __hmax2(__hmax2(h(raw.x), h(raw.y)), __hmax2(h(raw.z), h(raw.w)));
        return fmaxf(__low2float(m), __high2float(m));
    }
}

// A column and its logit; "better" orders by the logit, then by the lowest column.
struct Candidate {
    float v;
    int id;
};
__device__ __forceinline__ bool better(float v, int id, float v2, int id2) {
    return v > v2 || (v == v2 && id < id2);
}

// The running sums of a thread, or of several joined.
struct SoftmaxState {
    float m = -INFINITY, M = -INFINITY, s = 0.f, s1 = 0.f;
    // (a product of its own: fused into a difference it would not be the M that the terms saw)
    __device__ static float reference(float m, float c) { return __fmul_rn(m, c); }
    // whether terms are taken relative to the product M, rather than to m before it is scaled
    __device__ static bool usual(float M) { return fabsf(M) < 0x1p24f; }
    // log2 of the factor from one maximum to another, each as its terms see it; far below 0, 2^d
    // is 0 and the bound on d keeps products with it from being 0 times infinity
    __device__ static float step(float m, float M, float m2, float M2, float c) {
        const bool from = usual(M), to = usual(M2);
        return from && to ? M - M2 : from ? -fmaf(m2, c, -M) : to ? fmaf(m, c, -M2) : (m - m2) * c;
    }
    // raises the maximum to at least m2
    __device__ void raise(float m2, float c) {
        if (m2 > m) {
            const float M2 = reference(m2, c), d = step(m, M, m2, M2, c), f = exp2_approx(d);
            s1 = m == -INFINITY ? s1 : f * fmaf(s, fmaxf(d, -1000.f), s1);
            s *= f;
            m = m2;
            M = M2;
        }
    }
    // adds the N logits v, none of them above m, two at a time (N is 1 or even)
    template <int N>
    __device__ void add(const float *v, float c) {
        if (N > 1 && usual(M)) {
            F2 sum(s, 0.f), sum1(s1, 0.f);
            const F2 cc(c), MM(-M);
#pragma unroll
            for (int j = 0; j + 1 < N; j += 2) {
                const F2 t = fma(F2(v[j], v[j + 1]), cc, MM);
                const float2 x = t.both();
                const F2 e(exp2_approx(x.x), exp2_approx(x.y));
                sum = sum + e;
                sum1 = fma(e, t, sum1);
            }
            const float s1_new = sum1.sum();
            if (s1_new == s1_new) {
                s = sum.sum();
                s1 = s1_new;
                return;
            }
        }
        // a term of 0 times -infinity (a logit of -infinity), a NaN, or large logits
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float t = usual(M) ? fmaf(v[j], c, -M) : (v[j] - m) * c, e = exp2_approx(t);
            s += e;
            s1 = fmaf(e, fmaxf(t, -1000.f), s1);
        }
    }
    // joins the states of the warp's lanes: the largest maximum first, then plain sums relative to it
    __device__ void join_lanes(float c) {
        float m2 = m;
#pragma unroll
        for (int o = 16; o; o >>= 1) m2 = fmaxf(m2, __shfl_xor_sync(0xffffffffu, m2, o));
        if (m > -INFINITY) {  // otherwise s is 0, or NaN
            const float d = step(m, M, m2, reference(m2, c), c), f = exp2_approx(d);
            s1 = f * fmaf(s, fmaxf(d, -1000.f), s1);
            s *= f;
        }
        m = m2;
        M = reference(m2, c);
        s = warp_sum(s);
        s1 = warp_sum(s1);
    }
};

// Exchanges (v, id) with the lane `stride` away, keeping the better of the two
// where `keep_better` holds and the other elsewhere.
__device__ __forceinline__ void exchange(float &v, int &id, int stride, bool keep_better) {
    const float ov = __shfl_xor_sync(0xffffffffu, v, stride);
    const int oid = __shfl_xor_sync(0xffffffffu, id, stride);
    if (better(ov, oid, v, id) == keep_better) {
        v = ov;
        id = oid;
    }
}

// The best columns of a warp in order, lane i holding the i-th (none: -infinity).
struct WarpTop {
    float v = -INFINITY;
    int id = INT_MAX;
    // one more column
    __device__ void insert(float cv, int cid, int lane) {
        const bool ahead = better(v, id, cv, cid);
        const int pos = __popc(__ballot_sync(0xffffffffu, ahead));
        const float uv = __shfl_up_sync(0xffffffffu, v, 1);
        const int uid = __shfl_up_sync(0xffffffffu, id, 1);
        if (lane == pos) {
            v = cv;
            id = cid;
        } else if (lane > pos) {
            v = uv;
            id = uid;
        }
    }
    // one column a lane (none: -infinity): a bitonic sort of the new ones, the better halves of
    // both lists, and a bitonic merge
    __device__ void merge(float cv, int cid, int lane) {
#pragma unroll
        for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
            for (int stride = size >> 1; stride; stride >>= 1)
                exchange(cv, cid, stride, ((lane & stride) == 0) == ((lane & size) == 0));
        const float rv = __shfl_xor_sync(0xffffffffu, cv, 31);
        const int rid = __shfl_xor_sync(0xffffffffu, cid, 31);
        if (better(rv, rid, v, id)) {
            v = rv;
            id = rid;
        }
#pragma unroll
        for (int stride = 16; stride; stride >>= 1) exchange(v, id, stride, (lane & stride) == 0);
    }
};

// The k-th largest (k = 1 .. 32) of the lanes' values: a bitonic sort over lanes.
__device__ __forceinline__ float warp_kth_largest(float x, int k, int lane) {
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
        for (int stride = size >> 1; stride; stride >>= 1) {
            const float o = __shfl_xor_sync(0xffffffffu, x, stride);
            x = ((lane & stride) == 0) == ((lane & size) == 0) ? fmaxf(x, o) : fminf(x, o);
        }
    return __shfl_sync(0xffffffffu, x, k - 1);
}

// Columns that may be among a row's best, in any order, up to CAP of them.
template <int CAP>
struct Candidates {
    Candidate entry[CAP];
    int count;
    __device__ void push(float v, int id) {
        const int at = atomicAdd(&count, 1);  // their order does not matter
        if (at < CAP) entry[at] = {v, id};
    }
    // after a barrier: the `top` best into out, in order; an entry's place is the number of better ones
    __device__ void best(int top, Candidate *out) const {
        const int n = count;
        for (int i = threadIdx.x; i < n; i += blockDim.x) {
            const Candidate e = entry[i];
            int place = 0;
#pragma unroll 4
            for (int j = 0; j < n; ++j) place += better(entry[j].v, entry[j].id, e.v, e.id);
            if (place < top) out[place] = e;
        }
    }
};

constexpr int kTopBuffer = 512;  // columns; at least the 256 that a cluster's lists, or a block's warps', hold

// A cluster of gridDim.x blocks shares row blockIdx.y (+ gridDim.y, ...): each
// takes a run of 16-byte pieces; the last also the columns before the first
// and after the last aligned piece.  Block 0 joins the blocks' results through
// distributed shared memory.  Each thread copies its own pieces (U to a chunk,
// 16 elements) into its own places of a ring in shared memory, kLogprobDepth
// chunks ahead and on into the block's next row, so that memory is busy while a
// row's results are joined.
constexpr int kLogprobDepth = 4;
template <int DT>
constexpr int kLogprobPieces = 16 / Elem<DT>::VEC;
// bytes of the ring: a piece, and with a mask the two words that hold its bits
template <int DT, int THREADS, bool MASK>
constexpr int kLogprobRing = kLogprobDepth * kLogprobPieces<DT> * THREADS * (MASK ? 24 : 16);

// THREADS: 256, or fewer where a row gives a thread so few columns that what a
// row costs a warp beside them counts.  Registers for 1024 threads an SM (768
// where it takes more).
template <int DT, int THREADS, bool TOP, bool MASK>
__global__ void __launch_bounds__(THREADS, (TOP && MASK || DT == SGEMM_F32 && !TOP ? 768 : 1024) / THREADS)
    logprobs_kernel(const LogprobArgs a) {
    using E = Elem<DT>;
    using type = typename E::type;
    constexpr int VEC = E::VEC, WARPS = THREADS / 32, U = kLogprobPieces<DT>,
                  DEPTH = kLogprobDepth;
    extern __shared__ uint4 ring[];
    __shared__ float warp_state[3][WARPS];
    __shared__ float block_state[3];
    __shared__ Candidate block_list[TOP ? 32 : 1];
    __shared__ Candidates<TOP ? kTopBuffer : 1> found;
    __shared__ uint8_t again[TOP ? THREADS : 1];
    __shared__ int again_count;
    __shared__ float group_max[32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int parts = gridDim.x, part = blockIdx.x, log_parts = __ffs(parts) - 1;  // parts: a power of two
    const float c = a.scale * kLog2e;

    // a row as this block reads it: `head` columns before the first aligned piece, pieces [p0, p1)
    struct Row {
        const type *z;
        const int32_t *mask;
        int head, pieces, p0, p1;
    };
    auto row_of = [&](int64_t t) {
        Row r;
        r.z = static_cast<const type *>(a.z) + t * a.ldz;
        r.mask = MASK ? a.mask + t * a.ldm : nullptr;
        const int off = (int)((reinterpret_cast<uintptr_t>(r.z) & 15u) / sizeof(type));
        r.head = min(off ? VEC - off : 0, a.V);
        r.pieces = (a.V - r.head) / VEC;
        r.p0 = (int)((int64_t)r.pieces * part >> log_parts);
        r.p1 = (int)((int64_t)r.pieces * (part + 1) >> log_parts);
        return r;
    };
    // the chunk that is copied next: of row `ahead_t`, from piece `ahead_p` on
    int64_t ahead_t = blockIdx.y;
    Row ahead;
    int ahead_p = 0;
    auto next_row = [&](int64_t t) {
        for (ahead_t = t; ahead_t < a.T; ahead_t += gridDim.y) {
            ahead = row_of(ahead_t);
            ahead_p = ahead.p0;
            if (ahead.p0 < ahead.p1) break;
        }
    };
    auto copy = [&](int slot) {
        if (ahead_t < a.T) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int at = ahead_p + u * THREADS + (int)threadIdx.x, place = (slot * U + u) * THREADS + threadIdx.x;
                if (at < ahead.p1) {
                    cp_async_16(smem_addr(ring + place), ahead.z + ahead.head + (int64_t)at * VEC, 16);
                    if (MASK) {
                        const uint32_t to = smem_addr(reinterpret_cast<uint2 *>(ring + DEPTH * U * THREADS) + place);
                        const int w = (ahead.head + at * VEC) >> 5, last = (a.V - 1) >> 5;
                        cp_async_4(to, ahead.mask + w, 4);
                        cp_async_4(to + 4, ahead.mask + min(w + 1, last), 4);
                    }
                }
            }
            ahead_p += THREADS * U;
            if (ahead_p >= ahead.p1) next_row(ahead_t + gridDim.y);
        }
        cp_async_commit();
    };
    next_row(blockIdx.y);
#pragma unroll
    for (int s = 0; s < DEPTH; ++s) copy(s);
    int slot = 0;

    for (int64_t t = blockIdx.y; t < a.T; t += gridDim.y) {
        const Row row = row_of(t);
        const type *z = row.z;
        const int32_t *mask = row.mask;
        const int head = row.head, tail0 = head + row.pieces * VEC;

        SoftmaxState st;
        // adds the n columns v of this thread, -infinity where there is none; top: their largest
        auto add = [&](const float *v, float top, auto n_const) {
            constexpr int n = decltype(n_const)::value;
            st.raise(top, c);
            if (st.m == -INFINITY) {
#pragma unroll
                for (int j = 0; j < n; ++j)
                    if (v[j] != v[j]) st.s = v[j];
            } else {
                st.template add<n>(v, c);
            }
        };
        auto allowed = [&](int col) { return !MASK || (mask[col >> 5] >> (col & 31) & 1); };

        for (int p = row.p0; p < row.p1; p += THREADS * U) {
            cp_async_wait<DEPTH - 1>();
            float v[U * VEC], top = -INFINITY;
            // what lies outside the row, or is masked, is -infinity; neither test costs a whole chunk
            // of a call without a mask anything
            const bool whole = p + THREADS * U <= row.p1;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int place = (slot * U + u) * THREADS + threadIdx.x;
                const uint4 raw = ring[place];
                unpack16<DT>(raw, v + u * VEC);
                if (MASK || !whole) {
                    const int at = p + u * THREADS + (int)threadIdx.x;
                    uint32_t bits = ~0u;
                    if (MASK) {
                        const uint2 w = reinterpret_cast<const uint2 *>(ring + DEPTH * U * THREADS)[place];
                        bits = __funnelshift_r(w.x, w.y, (head + at * VEC) & 31);
                    }
                    if (at >= row.p1) bits = 0;
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        if (!(bits >> e & 1)) v[u * VEC + e] = -INFINITY;
                        top = fmaxf(top, v[u * VEC + e]);
                    }
                } else {
                    top = fmaxf(top, max16<DT>(raw));
                }
            }
            copy(slot);
            slot = slot + 1 == DEPTH ? 0 : slot + 1;
            add(v, top, std::integral_constant<int, U * VEC>{});
        }
        const float thread_max = st.m;  // of the thread's pieces
        // fewer than 2 * VEC columns lie outside the pieces: one a lane of the last block's first warp
        Candidate outside{-INFINITY, INT_MAX};
        if (part == parts - 1 && warp == 0 && lane < head + a.V - tail0) {
            const int col = lane < head ? lane : tail0 + lane - head;
            if (allowed(col)) outside = {E::to_float(z[col]), col};
            add(&outside.v, outside.v, std::integral_constant<int, 1>{});
        }

        if constexpr (TOP) {
            // At least `top` columns reach the top-th largest of the maxima of the block's 32 groups
            // of threads, so only threads whose own maximum does have columns to look at again: a
            // handful, unless many logits are equal.  Their pieces, one a lane, come from L2.
            float g = thread_max;
#pragma unroll
            for (int o = 32 / WARPS; o < 32; o <<= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
            if (lane < 32 / WARPS) group_max[warp * (32 / WARPS) + lane] = g;
            if (threadIdx.x == 0) found.count = again_count = 0;
            if (warp == 0) block_list[lane] = {-INFINITY, INT_MAX};
            __syncthreads();
            const float floor_v = warp_kth_largest(group_max[lane], a.top, lane);
            if (thread_max >= floor_v && thread_max > -INFINITY) again[atomicAdd(&again_count, 1)] = (uint8_t)threadIdx.x;
            if (outside.v >= floor_v && outside.v > -INFINITY) found.push(outside.v, outside.id);
            __syncthreads();
            // the columns of a piece
            auto columns = [&](int at, auto take) {
                const bool in = at < row.p1;
                const int col = head + at * VEC;
                float v[VEC];
                unpack16<DT>(in ? __ldg(reinterpret_cast<const uint4 *>(z + head) + at) : make_uint4(0, 0, 0, 0), v);
                const uint32_t bits = !in ? 0u : MASK ? mask_bits(mask, col, VEC, a.V) : ~0u;
#pragma unroll
                for (int e = 0; e < VEC; ++e) take((bits >> e & 1) && v[e] >= floor_v && v[e] > -INFINITY, v[e], col + e);
            };
            // all pieces of all those threads, one a thread
            const int n_again = again_count, per = (row.p1 - row.p0 + THREADS - 1) / THREADS;
            for (int i = threadIdx.x; i < n_again * per; i += THREADS)
                columns(row.p0 + again[i / per] + (i % per) * THREADS, [&](bool in, float v, int id) {
                    if (in) found.push(v, id);
                });
            __syncthreads();
            if (found.count > kTopBuffer) {
                // too many (equal logits): every warp keeps the best of its share in order instead
                WarpTop best;
                float last_v = -INFINITY;
                int last_id = INT_MAX;
                auto offer = [&](bool in, float v, int id) {
                    in = in && better(v, id, last_v, last_id);
                    unsigned who = __ballot_sync(0xffffffffu, in);
                    if (!who) return;
                    if (__popc(who) > 6) {
                        best.merge(in ? v : -INFINITY, in ? id : INT_MAX, lane);
                    } else {
                        for (; who; who &= who - 1) {
                            const int src = __ffs(who) - 1;
                            best.insert(__shfl_sync(0xffffffffu, v, src), __shfl_sync(0xffffffffu, id, src), lane);
                        }
                    }
                    last_v = __shfl_sync(0xffffffffu, best.v, a.top - 1);
                    last_id = __shfl_sync(0xffffffffu, best.id, a.top - 1);
                };
                for (int i = warp; i < n_again; i += WARPS)
                    for (int j = 0; j < per; j += 32)
                        columns(j + lane < per ? row.p0 + again[i] + (j + lane) * THREADS : row.p1, offer);
                offer(outside.v >= floor_v && outside.v > -INFINITY, outside.v, outside.id);
                __syncthreads();
                if (threadIdx.x == 0) found.count = 0;
                __syncthreads();
                if (lane < a.top && best.v > -INFINITY) found.push(best.v, best.id);
                __syncthreads();
            }
            found.best(a.top, block_list);
        }

        // ---- join the lanes, the warps, and the cluster's blocks
        st.join_lanes(c);
        if (lane == 0) {
            warp_state[0][warp] = st.m;
            warp_state[1][warp] = st.s;
            warp_state[2][warp] = st.s1;
        }
        __syncthreads();
        SoftmaxState all;
        if (warp == 0) {
            if (lane < WARPS) {
                all.m = warp_state[0][lane];
                all.M = SoftmaxState::reference(all.m, c);
                all.s = warp_state[1][lane];
                all.s1 = warp_state[2][lane];
            }
            all.join_lanes(c);
            if (parts > 1 && lane == 0) {
                block_state[0] = all.m;
                block_state[1] = all.s;
                block_state[2] = all.s1;
            }
        }
        if (parts > 1) {
            __syncthreads();
            cluster_sync();
            if (part == 0) {
                if (warp == 0) {
                    all = SoftmaxState{};
                    if (lane < parts) {
                        const uint32_t s = dsmem_map(smem_addr(block_state), (uint32_t)lane);
                        all.m = __uint_as_float(dsmem_ld_u32(s));
                        all.M = SoftmaxState::reference(all.m, c);
                        all.s = __uint_as_float(dsmem_ld_u32(s + 4));
                        all.s1 = __uint_as_float(dsmem_ld_u32(s + 8));
                    }
                    all.join_lanes(c);
                }
                if constexpr (TOP) {
                    if (threadIdx.x == 0) found.count = 0;
                    __syncthreads();
                    // no column below the largest of the lists' last can be among the best
                    float v = -INFINITY;
                    int id = INT_MAX;
                    if (warp < parts && lane < a.top) {
                        const uint32_t l = dsmem_map(smem_addr(&block_list[lane]), (uint32_t)warp);
                        v = __uint_as_float(dsmem_ld_u32(l));
                        id = (int)dsmem_ld_u32(l + 4);
                    }
                    if (lane == a.top - 1) group_max[warp] = v;
                    __syncthreads();
                    float floor_v = -INFINITY;
                    for (int w = 0; w < WARPS; ++w) floor_v = fmaxf(floor_v, group_max[w]);
                    if (v > -INFINITY && v >= floor_v) found.push(v, id);
                    __syncthreads();  // block 0's own list has been read before it is written
                    if (warp == 0) block_list[lane] = {-INFINITY, INT_MAX};
                    __syncthreads();
                    found.best(a.top, block_list);
                    __syncthreads();
                }
            }
        }
        if (part == 0 && warp == 0) {
            const bool none = all.m == -INFINITY && !(all.s != all.s);
            // ln of the sum relative to exactly m
            const float off = SoftmaxState::usual(all.M) ? -fmaf(all.m, c, -all.M) : 0.f;
            const float log_s = logf(all.s), log_sum = fmaf(kLn2, off, log_s);
            if (lane == 0) {
                if (a.lse) a.lse[t] = none ? -INFINITY : fmaf(all.m, a.scale, log_sum);
                if (a.entropy) a.entropy[t] = none ? 0.f : log_s - kLn2 * (all.s1 / all.s);
                if (a.logprob) {
                    const int64_t y = a.target[t];
                    float lp = 0.f;
                    if (y >= a.V) {
                        lp = NAN;
                    } else if (y >= 0) {
                        const float zy = allowed((int)y) ? E::to_float(z[y]) : -INFINITY;
                        lp = none ? -INFINITY : fmaf(zy - all.m, a.scale, -log_sum);
                    }
                    a.logprob[t] = lp;
                }
            }
            if constexpr (TOP) {
                if (lane < a.top) {
                    const Candidate e = block_list[lane];
                    const bool bad = all.s != all.s;
                    const bool has = e.v > -INFINITY && !bad;
                    a.top_logprob[t * a.top + lane] = bad ? NAN : has ? fmaf(e.v - all.m, a.scale, -log_sum) : -INFINITY;
                    a.top_id[t * a.top + lane] = has ? e.id : -1;
                }
            }
        }
        __syncthreads();
        if (parts > 1) cluster_sync();  // no block leaves, or starts another row, while block 0 reads its results
    }
}

struct LogprobGradArgs {
    int T, V;
    const void *z;
    int64_t ldz;
    float scale;
    const int32_t *mask;
    int64_t ldm;
    const int64_t *target;
    const float *lse, *entropy, *g_logprob, *g_entropy;
    void *dz;
    int64_t lddz;
};

// dz_j = scale (g ([j = y] - p_j) - g_H p_j (log p_j + H)) for the columns of a
// row: p_j (A + B log p_j) with A = -scale (g + g_H H), B = -scale g_H, and the
// target's scale g on top.
struct LogprobGradRow {
    float scale, lse, A, B, hit;
    int target;  // -1: none
    bool usual;  // what the packed path below takes
    // the lowest value that the packed path sees of 16-bit logits; -infinity counts as it
    template <int DT>
    static constexpr float kLowest = DT == SGEMM_F16 ? -65504.f : -1e30f;
    template <int DT>
    __device__ static LogprobGradRow load(const LogprobGradArgs &a, int64_t t) {
        LogprobGradRow r(a, t);
        // all from there down has p = 0, and B log p is a number
        const float logp = fmaf(kLowest<DT>, r.scale, -r.lse);
        r.usual = logp < -128.f && fabsf(r.B * logp) < 1e37f;
        return r;
    }
    __device__ LogprobGradRow(const LogprobGradArgs &a, int64_t t) {
        scale = a.scale;
        lse = a.lse[t];
        const int64_t y = a.target[t];
        float g = y >= 0 ? a.g_logprob[t] : 0.f;
        if (y >= a.V) g = NAN;
        target = y >= 0 && y < a.V ? (int)y : -1;
        const float gh = a.g_entropy ? a.g_entropy[t] : 0.f;
        A = -a.scale * (a.g_entropy ? fmaf(gh, a.entropy[t], g) : g);
        B = -a.scale * gh;
        hit = a.scale * g;
    }
    __device__ float one(float z) const {
        // p below 2^-126 counts: its product with B log p may be above.  p = 0 leaves nothing of it
        // (log p may be -infinity there).
        const float logp = fmaf(z, scale, -lse), p = exp2_small(logp * kLog2e);
        return lse == -INFINITY ? 0.f : p * fmaf(B, fmaxf(logp, -1000.f), A);
    }
    // the N columns from `col` on; bits: which of them the mask allows
    template <int N>
    __device__ void apply(float *v, uint32_t bits, int col) const {
        const int at = target - col;
        const bool hits = at >= 0 && at < N;
        float target_z = -INFINITY;
        if (hits)
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (at == e) target_z = v[e];
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = bits >> e & 1 ? one(v[e]) : 0.f;
        if (hits && (bits >> at & 1) && target_z > -INFINITY && lse > -INFINITY)
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (at == e) v[e] += hit;
    }
    // the same for 8 columns of 16 bits, in packed pairs.  scale z - lse is rounded once, after they
    // cancel: the entropy's gradient needs log p itself where p is near 1.  The exponential is
    // taken 2^24 times too large, so that p counts down to 2^-150.
    template <int DT>
    __device__ uint4 apply16(uint4 raw, uint32_t bits, int col) const {
        float v[8];
        if (!usual || (unsigned)(target - col) < 8u) {
            unpack16<DT>(raw, v);
            apply<8>(v, bits, col);
            return pack16<DT>(v);
        }
        // no -infinity, whose logarithm times a p of 0 would not be 0
        uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (DT == SGEMM_BF16) {
                const __nv_bfloat162 m = __hmax2(*reinterpret_cast<__nv_bfloat162 *>(&w[i]), __float2bfloat162_rn(kLowest<DT>));
                w[i] = *reinterpret_cast<const uint32_t *>(&m);
            } else {
                const __half2 m = __hmax2(*reinterpret_cast<__half2 *>(&w[i]), __float2half2_rn(kLowest<DT>));
                w[i] = *reinterpret_cast<const uint32_t *>(&m);
            }
        }
        unpack16<DT>(make_uint4(w[0], w[1], w[2], w[3]), v);
        const F2 c(scale), off(-lse), a(A * 0x1p-24f), b(B * 0x1p-24f), log2e(kLog2e), up(24.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const F2 logp = fma(F2(v[2 * i], v[2 * i + 1]), c, off);
            const float2 t = fma(logp, log2e, up).both();
            const float2 d = (F2(exp2_approx(t.x), exp2_approx(t.y)) * fma(b, logp, a)).both();
            v[2 * i] = d.x;
            v[2 * i + 1] = d.y;
        }
        uint4 out = pack16<DT>(v);
        if (bits != 0xffu) {
            uint32_t *o = &out.x;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[i] &= (bits >> (2 * i) & 1 ? 0xffffu : 0u) | (bits >> (2 * i + 1) & 1 ? 0xffff0000u : 0u);
        }
        return out;
    }
};

// blockIdx.y (+ gridDim.y, ...): rows; blockIdx.x: runs of THREADS * U pieces
// of VW elements.  Every element is read before the same thread writes it, so
// dz may be the logits.
template <int DT, int VW, int THREADS, int U, bool MASK>
__global__ void __launch_bounds__(THREADS) logprobs_grad_kernel(const LogprobGradArgs a) {
    using E = Elem<DT>;
    using type = typename E::type;
    for (int64_t t = blockIdx.y; t < a.T; t += gridDim.y) {
        const type *z = static_cast<const type *>(a.z) + t * a.ldz;
        type *dz = static_cast<type *>(a.dz) + t * a.lddz;
        const int32_t *mask = MASK ? a.mask + t * a.ldm : nullptr;
        const LogprobGradRow row = LogprobGradRow::load<DT>(a, t);
        // 16-byte pieces need both rows at the same distance from a 16-byte boundary
        const int off = VW > 1 ? (int)((reinterpret_cast<uintptr_t>(z) & 15u) / sizeof(type)) : 0;
        const int head = min(off ? VW - off : 0, a.V);
        const int pieces = (a.V - head) / VW;
        const int tail0 = head + pieces * VW;
        const int base = blockIdx.x * (THREADS * U);
        using P = Piece<DT, VW>;
        typename P::raw raw[U];
        uint32_t bits[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = base + u * THREADS + (int)threadIdx.x;
            if (at < pieces) raw[u] = P::load(z + head + (int64_t)at * VW);
            bits[u] = ~0u;
            if (MASK && at < pieces) bits[u] = mask_bits(mask, head + at * VW, VW, a.V);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = base + u * THREADS + (int)threadIdx.x;
            if (at >= pieces) continue;
            const int col = head + at * VW;
            if constexpr (VW == 8) {
                *reinterpret_cast<uint4 *>(dz + col) = row.template apply16<DT>(raw[u], bits[u] & 0xffu, col);
            } else {
                float v[VW];
                P::unpack(raw[u], v);
                row.template apply<VW>(v, bits[u], col);
                P::store(dz + col, v);
            }
        }
        if (VW > 1 && blockIdx.x == gridDim.x - 1 && (int)threadIdx.x < head + a.V - tail0) {
            const int col = (int)threadIdx.x < head ? (int)threadIdx.x : tail0 + (int)threadIdx.x - head;
            const bool allowed = !MASK || (mask[col >> 5] >> (col & 31) & 1);
            float v = E::to_float(z[col]);
            row.template apply<1>(&v, allowed, col);
            dz[col] = E::from_float(v);
        }
    }
}

}  // namespace sgemm
