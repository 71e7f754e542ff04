// Log probabilities of given columns, entropy, log-sum-exp and the most likely
// columns of rows of logits, in one pass over them; and the gradient.
//
// With m the largest logit seen, t_j = (z_j - m) scale log2(e), the pass keeps
//     s = sum 2^t_j   and   s1 = sum 2^t_j t_j,
// which a larger m turns into f s and f (s1 + s d), d = (m - m') scale log2(e),
// f = 2^d.  At the end lse = scale m + ln s, entropy = ln s - ln 2 s1 / s, and
// log p_y = scale (z_y - m) - ln s.  The difference z_j - m is taken before the
// scale, so that logits of the type's lowest value stay finite.
//
// Each warp keeps the `top` best columns it has met as a list over its lanes,
// best first.  A chunk whose largest logits do not reach the list's last entry
// costs one comparison a lane; otherwise the columns of the lanes that do are
// looked at, 32 at a time, one a lane.  After 1, 2, 4, ... chunks the block also
// takes the top-th largest of the maxima of 32 groups of its threads, which
// every column has to reach from then on: a warp alone would let eight times
// as many through.
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

// Bits of the mask's row for columns c .. c + n - 1 (n <= 8), lowest first;
// columns from V on read as 0.
__device__ __forceinline__ uint32_t mask_bits(const int32_t *row, int c, int n, int V) {
    const int w = c >> 5, s = c & 31;
    uint32_t lo = (uint32_t)row[w], hi = 0;
    if (s + n > 32 && (w + 1) * 32 < V) hi = (uint32_t)row[w + 1];
    return __funnelshift_r(lo, hi, s);
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
    float m = -INFINITY, s = 0.f, s1 = 0.f;
    // raises the maximum to at least m2; where d is far below 0, 2^d is 0 and the bound on d
    // keeps the product from being 0 times infinity
    __device__ void raise(float m2, float c) {
        if (m2 > m) {
            const float d = (m - m2) * c, f = exp2_approx(d);
            s1 = m == -INFINITY ? s1 : f * fmaf(s, fmaxf(d, -1000.f), s1);
            s *= f;
            m = m2;
        }
    }
    // adds the n logits v, none of them above m (finite or +infinity), two at a time
    template <int N>
    __device__ void add(const float *v, float c) {
        if constexpr (N % 2 == 0) {
            const uint64_t mm = f32x2_dup(-m), cc = f32x2_dup(c);
            uint64_t sum = f32x2_pair(s, 0.f), sum1 = f32x2_pair(s1, 0.f);
#pragma unroll
            for (int j = 0; j < N; j += 2) {
                const uint64_t t = f32x2_mul(f32x2_add(f32x2_pair(v[j], v[j + 1]), mm), cc);
                const float2 x = f32x2_unpack(t);
                const uint64_t e = f32x2_pair(exp2_approx(x.x), exp2_approx(x.y));
                sum = f32x2_add(sum, e);
                f32x2_fma(sum1, e, t);
            }
            const float2 a = f32x2_unpack(sum), b = f32x2_unpack(sum1);
            const float s_new = a.x + a.y, s1_new = b.x + b.y;
            if (s1_new == s1_new) {
                s = s_new;
                s1 = s1_new;
                return;
            }
        }
        // a term of 0 times -infinity (a logit of -infinity), or a NaN
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float t = (v[j] - m) * c, e = exp2_approx(t);
            s += e;
            s1 = fmaf(e, fmaxf(t, -1000.f), s1);
        }
    }
    __device__ void join(float m2, float s2, float s12, float c) {
        if (m2 == -INFINITY) {
            s += s2;  // 0, or NaN
            return;
        }
        raise(m2, c);
        const float d = (m2 - m) * c, f = exp2_approx(d);
        s1 = fmaf(f, fmaf(s2, fmaxf(d, -1000.f), s12), s1);
        s = fmaf(s2, f, s);
    }
    // joins the states of 2 * FROM lanes, in an order that the lanes' numbers fix
    template <int FROM>
    __device__ void join_lanes(float c) {
#pragma unroll
        for (int o = FROM; o; o >>= 1) {
            const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o),
                        s12 = __shfl_xor_sync(0xffffffffu, s1, o);
            join(m2, s2, s12, c);
        }
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

// Joins the block's THREADS entries, one a thread, which are lists in order
// with `top` entries each: `top` best into out, in order.  No entry below the
// largest of the lists' last entries can be among them (that list alone has
// `top` better ones), so only those that reach it are compared with each
// other: an entry's place is the number of better ones.
template <int THREADS>
struct TopJoin {
    Candidate entry[THREADS];
    float last[THREADS / 32];
    int count;
    __device__ void run(float v, int id, int top, Candidate *out) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        if (lane == top - 1) last[warp] = v;
        if (threadIdx.x == 0) count = 0;
        if (threadIdx.x < 32) out[threadIdx.x] = {-INFINITY, INT_MAX};
        __syncthreads();
        float floor_v = -INFINITY;
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) floor_v = fmaxf(floor_v, last[w]);
        const bool in = lane < top && v > -INFINITY && v >= floor_v;
        if (in) entry[atomicAdd(&count, 1)] = {v, id};  // their order does not matter
        __syncthreads();
        if (in) {
            int place = 0;
            for (int i = 0, n = count; i < n; ++i) place += better(entry[i].v, entry[i].id, v, id);
            if (place < top) out[place] = {v, id};
        }
        __syncthreads();
    }
};

constexpr int kLogprobThreads = 256;

// A cluster of gridDim.x blocks shares row blockIdx.y (+ gridDim.y, ...): each
// takes a run of 16-byte pieces; the last also the columns before the first
// and after the last aligned piece.  Block 0 joins the blocks' results through
// distributed shared memory.  A thread loads U pieces ahead of those it adds up.
template <int DT, int U, bool TOP, bool MASK>
__global__ void __launch_bounds__(kLogprobThreads, U * Elem<DT>::VEC == 16 ? 3 : 2) logprobs_kernel(const LogprobArgs a) {
    using E = Elem<DT>;
    using type = typename E::type;
    constexpr int VEC = E::VEC, THREADS = kLogprobThreads, WARPS = THREADS / 32;
    __shared__ float warp_state[3][WARPS];
    __shared__ float block_state[3];
    __shared__ Candidate block_list[TOP ? 32 : 1];
    __shared__ TopJoin<TOP ? THREADS : 32> top_join;
    // a warp's columns on their way to its list, and the lanes that they come from
    __shared__ __align__(16) float columns[TOP ? WARPS : 1][TOP ? 32 * U * VEC : 4];
    __shared__ uint8_t from_lane[TOP ? WARPS : 1][32];
    __shared__ float group_max[2][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int parts = gridDim.x, part = blockIdx.x;
    const float c = a.scale * kLog2e;

    for (int64_t t = blockIdx.y; t < a.T; t += gridDim.y) {
        const type *z = static_cast<const type *>(a.z) + t * a.ldz;
        const int32_t *mask = MASK ? a.mask + t * a.ldm : nullptr;
        const int off = (int)((reinterpret_cast<uintptr_t>(z) & 15u) / sizeof(type));
        const int head = min(off ? VEC - off : 0, a.V);
        const int pieces = (a.V - head) / VEC;
        const int tail0 = head + pieces * VEC;
        const int p0 = (int)((int64_t)pieces * part / parts), p1 = (int)((int64_t)pieces * (part + 1) / parts);
        const uint4 *body = reinterpret_cast<const uint4 *>(z + head);

        SoftmaxState st;
        WarpTop best;
        // a column joins the warp's list if it is better than the list's last entry, and reaches
        // floor_v (which `top` of the row's columns are known to reach)
        float last_v = -INFINITY, floor_v = -INFINITY;
        int last_id = INT_MAX;
        // adds the columns v[0 .. n) of this thread, -infinity where there is none; column i of
        // lane l's has number col(l, i).  round: how many chunks the block has behind it, or -1
        // where only one warp is here
        auto chunk = [&](const float *v, auto n_const, int round, auto col) {
            constexpr int n = decltype(n_const)::value;
            float top = v[0];
#pragma unroll
            for (int j = 1; j < n; ++j) top = fmaxf(top, v[j]);
            st.raise(top, c);
            if (st.m == -INFINITY) {
#pragma unroll
                for (int j = 0; j < n; ++j)
                    if (v[j] != v[j]) st.s = v[j];
            } else {
                st.template add<n>(v, c);
            }
            if constexpr (TOP) {
                if ((round & (round + 1)) == 0 && round >= 0) {
                    // after 1, 2, 4, ... chunks: `top` columns reach the top-th largest of the
                    // maxima of the block's 32 groups of threads
                    float g = st.m;
#pragma unroll
                    for (int o = 32 / WARPS; o < 32; o <<= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
                    float *group = group_max[__popc(round) & 1];
                    if (lane < 32 / WARPS) group[warp * (32 / WARPS) + lane] = g;
                    __syncthreads();
                    floor_v = fmaxf(floor_v, warp_kth_largest(group[lane], a.top, lane));
                }
                const bool reaches = top >= fmaxf(last_v, floor_v) && top > -INFINITY;
                const unsigned reach = __ballot_sync(0xffffffffu, reaches);
                if (reach) {
                    // the columns of the lanes that reach it, one a lane, 32 at a time
                    if (reaches) {
                        const int rank = __popc(reach & ((1u << lane) - 1));
                        from_lane[warp][rank] = (uint8_t)lane;
                        float *to = &columns[warp][rank * n];
                        if constexpr (n % 4 == 0) {
#pragma unroll
                            for (int j = 0; j < n; j += 4)
                                *reinterpret_cast<float4 *>(to + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
                        } else {
#pragma unroll
                            for (int j = 0; j < n; ++j) to[j] = v[j];
                        }
                    }
                    __syncwarp();
                    for (int i = 0, count = __popc(reach) * n; i < count; i += 32) {
                        Candidate e{-INFINITY, INT_MAX};
                        if (i + lane < count) {
                            e.v = columns[warp][i + lane];
                            e.id = col(from_lane[warp][(i + lane) / n], (i + lane) % n);
                        }
                        const bool in = e.v >= floor_v && e.v > -INFINITY && better(e.v, e.id, last_v, last_id);
                        unsigned who = __ballot_sync(0xffffffffu, in);
                        if (!who) continue;
                        if (__popc(who) > 6) {
                            best.merge(in ? e.v : -INFINITY, in ? e.id : INT_MAX, lane);
                        } else {
                            for (; who; who &= who - 1) {
                                const int src = __ffs(who) - 1;
                                best.insert(__shfl_sync(0xffffffffu, e.v, src), __shfl_sync(0xffffffffu, e.id, src), lane);
                            }
                        }
                        last_v = __shfl_sync(0xffffffffu, best.v, a.top - 1);
                        last_id = __shfl_sync(0xffffffffu, best.id, a.top - 1);
                    }
                    __syncwarp();
                }
            }
        };
        auto allowed = [&](int col) { return !MASK || (mask[col >> 5] >> (col & 31) & 1); };

        auto load = [&](int p, uint4(&raw)[U], uint32_t(&bits)[U]) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int at = p + u * THREADS + (int)threadIdx.x;
                if (at < p1) raw[u] = __ldg(body + at);
                if (MASK && at < p1) bits[u] = mask_bits(mask, head + at * VEC, VEC, a.V);
            }
        };
        uint4 raw[U];
        uint32_t bits[U];
        load(p0, raw, bits);
        int round = 0;
        for (int p = p0; p < p1; p += THREADS * U) {
            float v[U * VEC];
            const bool whole = p + THREADS * U <= p1;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                unpack16<DT>(raw[u], v + u * VEC);
                if (MASK) {
#pragma unroll
                    for (int e = 0; e < VEC; ++e)
                        if (!(bits[u] >> e & 1)) v[u * VEC + e] = -INFINITY;
                }
                if (!whole && p + u * THREADS + (int)threadIdx.x >= p1) {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) v[u * VEC + e] = -INFINITY;
                }
            }
            if (p + THREADS * U < p1) load(p + THREADS * U, raw, bits);
            chunk(v, std::integral_constant<int, U * VEC>{}, round++, [&](int src, int i) {
                return head + (p + (i / VEC) * THREADS + warp * 32 + src) * VEC + i % VEC;
            });
        }
        if (part == parts - 1) {
            // fewer than 2 * VEC columns outside the pieces: one a lane of the first warp
            const int outside = head + a.V - tail0;
            if (warp == 0 && outside > 0) {
                auto column = [&](int l, int) { return l < head ? l : tail0 + l - head; };
                float v = -INFINITY;
                if (lane < outside && allowed(column(lane, 0))) v = E::to_float(z[column(lane, 0)]);
                chunk(&v, std::integral_constant<int, 1>{}, -1, column);
            }
        }

        // ---- join the lanes, the warps, and the cluster's blocks
        st.template join_lanes<16>(c);
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
                all.s = warp_state[1][lane];
                all.s1 = warp_state[2][lane];
            }
            all.template join_lanes<WARPS / 2>(c);
            if (parts > 1 && lane == 0) {
                block_state[0] = all.m;
                block_state[1] = all.s;
                block_state[2] = all.s1;
            }
        }
        if constexpr (TOP) top_join.run(best.v, best.id, a.top, block_list);
        if (parts > 1) {
            __syncthreads();
            cluster_sync();
            if (part == 0) {
                if (warp == 0) {
                    all = SoftmaxState{};
                    if (lane < parts) {
                        const uint32_t s = dsmem_map(smem_addr(block_state), (uint32_t)lane);
                        all.m = __uint_as_float(dsmem_ld_u32(s));
                        all.s = __uint_as_float(dsmem_ld_u32(s + 4));
                        all.s1 = __uint_as_float(dsmem_ld_u32(s + 8));
                    }
                    all.template join_lanes<4>(c);
                }
                if constexpr (TOP) {
                    Candidate e{-INFINITY, INT_MAX};
                    if (warp < parts) {
                        const uint32_t l = dsmem_map(smem_addr(&block_list[lane]), (uint32_t)warp);
                        e.v = __uint_as_float(dsmem_ld_u32(l));
                        e.id = (int)dsmem_ld_u32(l + 4);
                    }
                    __syncthreads();  // block 0's own list has been read before it is written
                    top_join.run(e.v, e.id, a.top, block_list);
                }
            }
        }
        if (part == 0 && warp == 0) {
            all.m = __shfl_sync(0xffffffffu, all.m, 0);
            all.s = __shfl_sync(0xffffffffu, all.s, 0);
            const bool none = all.m == -INFINITY && !(all.s != all.s);
            const float log_s = logf(all.s);
            if (lane == 0) {
                if (a.lse) a.lse[t] = none ? -INFINITY : fmaf(all.m, a.scale, log_s);
                if (a.entropy) a.entropy[t] = none ? 0.f : log_s - kLn2 * (all.s1 / all.s);
                if (a.logprob) {
                    const int64_t y = a.target[t];
                    float lp = 0.f;
                    if (y >= a.V) {
                        lp = NAN;
                    } else if (y >= 0) {
                        const float zy = allowed((int)y) ? E::to_float(z[y]) : -INFINITY;
                        lp = none ? -INFINITY : fmaf(zy - all.m, a.scale, -log_s);
                    }
                    a.logprob[t] = lp;
                }
            }
            if constexpr (TOP) {
                if (lane < a.top) {
                    const Candidate e = block_list[lane];
                    const bool bad = all.s != all.s;
                    const bool has = e.v > -INFINITY && !bad;
                    a.top_logprob[t * a.top + lane] = bad ? NAN : has ? fmaf(e.v - all.m, a.scale, -log_s) : -INFINITY;
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

// dz_j = scale (g ([j = y] - p_j) - g_H p_j (log p_j + H)) for one column:
// p_j (A + B log p_j) with A = -scale (g + g_H H), B = -scale g_H, and the
// target's scale g on top.
struct LogprobGradRow {
    float scale, lse, A, B, hit;
    int64_t target;
    __device__ LogprobGradRow(const LogprobGradArgs &a, int64_t t) {
        scale = a.scale;
        lse = a.lse[t];
        target = a.target[t];
        float g = target >= 0 ? a.g_logprob[t] : 0.f;
        if (target >= a.V) g = NAN;
        const float gh = a.g_entropy ? a.g_entropy[t] : 0.f;
        A = -a.scale * (a.g_entropy ? fmaf(gh, a.entropy[t], g) : g);
        B = -a.scale * gh;
        hit = a.scale * g;
    }
    // the N columns from `col` on; bits: which of them the mask allows
    template <int N>
    __device__ void apply(float *v, uint32_t bits, int col) const {
        const bool near = target >= col && target < (int64_t)col + N;
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const float logp = fmaf(v[e], scale, -lse), p = exp2_approx(logp * kLog2e);
            // p = 0 leaves nothing of B log p (log p may be -infinity there)
            float d = p * fmaf(B, fmaxf(logp, -1000.f), A);
            if (near && target - col == e && v[e] > -INFINITY) d += hit;
            v[e] = !(bits >> e & 1) ? 0.f : d;
        }
        if (lse == -INFINITY) {
#pragma unroll
            for (int e = 0; e < N; ++e) v[e] = 0.f;
        }
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
        const LogprobGradRow row(a, t);
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
            float v[VW];
            P::unpack(raw[u], v);
            const int col = head + at * VW;
            row.template apply<VW>(v, bits[u], col);
            P::store(dz + col, v);
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
