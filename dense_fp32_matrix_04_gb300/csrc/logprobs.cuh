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
// costs one comparison a lane; otherwise its columns are first held to the
// top-th largest of the 32 lanes' maxima (at least `top` columns reach that),
// and those left are inserted one by one.
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

// The running sums of a thread.
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
    __device__ void add(float z, float c) {
        const float t = (z - m) * c, e = exp2_approx(t);
        s += e;
        s1 = fmaf(e, fmaxf(t, -1000.f), s1);  // as in raise()
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
};

// The `top` best columns of a warp, lane i holding the i-th (none: -infinity).
struct WarpTop {
    float v = -INFINITY;
    int id = INT_MAX;
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
};

// The k-th largest (k = 1 .. 32) of the lanes' values: a bitonic sort over lanes.
__device__ __forceinline__ float warp_kth_largest(float x, int k, int lane) {
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
        for (int stride = size >> 1; stride; stride >>= 1) {
            const float o = __shfl_xor_sync(0xffffffffu, x, stride);
            const bool down = (lane & size) == 0 || size == 32;   // this run sorts from large to small
            const bool lower = (lane & stride) == 0;
            x = down == lower ? fmaxf(x, o) : fminf(x, o);
        }
    return __shfl_sync(0xffffffffu, x, k - 1);
}

constexpr int kTopBuffer = 64;  // columns a warp collects before it inserts them

// A cluster of gridDim.x blocks shares row blockIdx.y (+ gridDim.y, ...): each
// takes a run of 16-byte pieces; the last also the columns before the first
// and after the last aligned piece.  Block 0 joins the blocks' results through
// distributed shared memory.
template <int DT, int THREADS, int U, bool TOP>
__global__ void __launch_bounds__(THREADS) logprobs_kernel(const LogprobArgs a) {
    using E = Elem<DT>;
    using type = typename E::type;
    constexpr int VEC = E::VEC, WARPS = THREADS / 32;
    __shared__ float warp_state[3][WARPS];
    __shared__ float block_state[3];
    __shared__ Candidate lists[TOP ? WARPS : 1][32];
    __shared__ Candidate block_list[TOP ? 32 : 1];
    __shared__ Candidate buffer[TOP ? WARPS : 1][TOP ? kTopBuffer : 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int parts = gridDim.x, part = blockIdx.x;
    const float c = a.scale * kLog2e;

    for (int64_t t = blockIdx.y; t < a.T; t += gridDim.y) {
        const type *z = static_cast<const type *>(a.z) + t * a.ldz;
        const int32_t *mask = a.mask ? a.mask + t * a.ldm : nullptr;
        const int off = (int)((reinterpret_cast<uintptr_t>(z) & 15u) / sizeof(type));
        const int head = min(off ? VEC - off : 0, a.V);
        const int pieces = (a.V - head) / VEC;
        const int tail0 = head + pieces * VEC;
        const int p0 = (int)((int64_t)pieces * part / parts), p1 = (int)((int64_t)pieces * (part + 1) / parts);
        const uint4 *body = reinterpret_cast<const uint4 *>(z + head);

        SoftmaxState st;
        WarpTop best;
        // the columns v[0 .. n) of this thread, column j at col(j); -infinity where there is none
        auto chunk = [&](const float *v, auto n_const, auto col) {
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
#pragma unroll
                for (int j = 0; j < n; ++j) st.add(v[j], c);
            }
            if constexpr (TOP) {
                const float last_v = __shfl_sync(0xffffffffu, best.v, a.top - 1);
                const unsigned reach = __ballot_sync(0xffffffffu, top >= last_v && top > -INFINITY);
                if (reach) {
                    const int last_id = __shfl_sync(0xffffffffu, best.id, a.top - 1);
                    float floor_v = -INFINITY;
                    if (__popc(reach) > a.top) floor_v = warp_kth_largest(top, a.top, lane);
                    uint32_t keep = 0;
#pragma unroll
                    for (int j = 0; j < n; ++j)
                        if (v[j] >= floor_v && v[j] > -INFINITY && better(v[j], col(j), last_v, last_id)) keep |= 1u << j;
                    int at = __popc(keep), total;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const int up = __shfl_up_sync(0xffffffffu, at, o);
                        if (lane >= o) at += up;
                    }
                    total = __shfl_sync(0xffffffffu, at, 31);
                    at -= __popc(keep);
                    for (int from = 0; from < total; from += kTopBuffer) {
                        int k = at;
#pragma unroll
                        for (int j = 0; j < n; ++j)
                            if (keep >> j & 1) {
                                if (k >= from && k < from + kTopBuffer) buffer[warp][k - from] = {v[j], col(j)};
                                ++k;
                            }
                        __syncwarp();
                        const int count = min(kTopBuffer, total - from);
                        for (int i = 0; i < count; ++i) {
                            const Candidate e = buffer[warp][i];
                            const float lv = __shfl_sync(0xffffffffu, best.v, a.top - 1);
                            const int li = __shfl_sync(0xffffffffu, best.id, a.top - 1);
                            if (better(e.v, e.id, lv, li)) best.insert(e.v, e.id, lane);
                        }
                        __syncwarp();
                    }
                }
            }
        };

        for (int p = p0; p < p1; p += THREADS * U) {
            uint4 raw[U];
            uint32_t bits[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int at = p + u * THREADS + (int)threadIdx.x;
                if (at < p1) raw[u] = body[at];
                bits[u] = at < p1 ? ~0u : 0u;
                if (mask && at < p1) bits[u] = mask_bits(mask, head + at * VEC, VEC, a.V);
            }
            float v[U * VEC];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                unpack16<DT>(raw[u], v + u * VEC);
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    if (!(bits[u] >> e & 1)) v[u * VEC + e] = -INFINITY;
            }
            chunk(v, std::integral_constant<int, U * VEC>{}, [&](int j) {
                return head + (p + (j / VEC) * THREADS + (int)threadIdx.x) * VEC + j % VEC;
            });
        }
        if (part == parts - 1) {
            // fewer than 2 * VEC columns outside the pieces: one a thread
            const int outside = head + a.V - tail0;
            float v = -INFINITY;
            int col = INT_MAX;
            if ((int)threadIdx.x < outside) {
                col = (int)threadIdx.x < head ? (int)threadIdx.x : tail0 + (int)threadIdx.x - head;
                if (!mask || (mask[col >> 5] >> (col & 31) & 1)) v = E::to_float(z[col]);
            }
            if (warp == 0 && outside > 0) chunk(&v, std::integral_constant<int, 1>{}, [&](int) { return col; });
        }

        // ---- join the lanes, the warps, and the cluster's blocks
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const float m2 = __shfl_xor_sync(0xffffffffu, st.m, o), s2 = __shfl_xor_sync(0xffffffffu, st.s, o),
                        s12 = __shfl_xor_sync(0xffffffffu, st.s1, o);
            st.join(m2, s2, s12, c);
        }
        if (lane == 0) {
            warp_state[0][warp] = st.m;
            warp_state[1][warp] = st.s;
            warp_state[2][warp] = st.s1;
        }
        if constexpr (TOP) {
            lists[warp][lane] = lane < a.top ? Candidate{best.v, best.id} : Candidate{-INFINITY, INT_MAX};
            if (warp == 0) block_list[lane] = {-INFINITY, INT_MAX};
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            SoftmaxState all;
            for (int w = 0; w < WARPS; ++w) all.join(warp_state[0][w], warp_state[1][w], warp_state[2][w], c);
            block_state[0] = all.m;
            block_state[1] = all.s;
            block_state[2] = all.s1;
        }
        if constexpr (TOP) {
            // an entry's place in the block's list is the number of better entries
            const Candidate e = lists[warp][lane];
            if (e.v > -INFINITY) {
                int place = 0;
                for (int w = 0; w < WARPS; ++w)
                    for (int i = 0; i < a.top; ++i) {
                        const Candidate o = lists[w][i];
                        if (!better(o.v, o.id, e.v, e.id)) break;  // the lists are in order
                        ++place;
                    }
                if (place < a.top) block_list[place] = e;
            }
        }
        if (parts > 1) cluster_sync();
        else __syncthreads();
        if (part == 0 && warp == 0) {
            SoftmaxState all;
            WarpTop joined;
            for (int b = 0; b < parts; ++b) {
                const uint32_t s = parts > 1 ? dsmem_map(smem_addr(block_state), (uint32_t)b) : 0;
                float m2, s2, s12;
                if (parts > 1) {
                    m2 = __uint_as_float(dsmem_ld_u32(s));
                    s2 = __uint_as_float(dsmem_ld_u32(s + 4));
                    s12 = __uint_as_float(dsmem_ld_u32(s + 8));
                } else {
                    m2 = block_state[0];
                    s2 = block_state[1];
                    s12 = block_state[2];
                }
                all.join(m2, s2, s12, c);
                if constexpr (TOP) {
                    float cv;
                    int ci;
                    if (parts > 1) {
                        const uint32_t l = dsmem_map(smem_addr(&block_list[lane]), (uint32_t)b);
                        cv = __uint_as_float(dsmem_ld_u32(l));
                        ci = (int)dsmem_ld_u32(l + 4);
                    } else {
                        cv = block_list[lane].v;
                        ci = block_list[lane].id;
                    }
                    if (b == 0) {
                        joined.v = cv;
                        joined.id = ci;
                    } else {
                        for (int i = 0; i < a.top; ++i) {
                            const float ev = __shfl_sync(0xffffffffu, cv, i);
                            const int ei = __shfl_sync(0xffffffffu, ci, i);
                            const float lv = __shfl_sync(0xffffffffu, joined.v, a.top - 1);
                            const int li = __shfl_sync(0xffffffffu, joined.id, a.top - 1);
                            if (!(ev > -INFINITY) || !better(ev, ei, lv, li)) break;
                            joined.insert(ev, ei, lane);
                        }
                    }
                }
            }
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
                        const bool allowed = !mask || (mask[y >> 5] >> (y & 31) & 1);
                        const float zy = allowed ? E::to_float(z[y]) : -INFINITY;
                        lp = none ? -INFINITY : fmaf(zy - all.m, a.scale, -log_s);
                    }
                    a.logprob[t] = lp;
                }
            }
            if constexpr (TOP) {
                if (lane < a.top) {
                    const bool bad = all.s != all.s;
                    const bool has = joined.v > -INFINITY && !bad;
                    a.top_logprob[t * a.top + lane] =
                        bad ? NAN : has ? fmaf(joined.v - all.m, a.scale, -log_s) : -INFINITY;
                    a.top_id[t * a.top + lane] = has ? joined.id : -1;
                }
            }
        }
        if (parts > 1) cluster_sync();
        else __syncthreads();
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
    __device__ float operator()(float z, bool allowed, int64_t col) const {
        if (!allowed || lse == -INFINITY) return 0.f;
        const float logp = fmaf(z, scale, -lse), p = exp2_approx(logp * kLog2e);
        // p = 0 leaves nothing of B log p (log p may be -infinity there)
        const float d = p * fmaf(B, fmaxf(logp, -1000.f), A);
        return col == target && z > -INFINITY ? d + hit : d;
    }
};

// blockIdx.y (+ gridDim.y, ...): rows; blockIdx.x: runs of THREADS * U pieces
// of VW elements.  Every element is read before the same thread writes it, so
// dz may be the logits.
template <int DT, int VW, int THREADS, int U>
__global__ void __launch_bounds__(THREADS) logprobs_grad_kernel(const LogprobGradArgs a) {
    using E = Elem<DT>;
    using type = typename E::type;
    for (int64_t t = blockIdx.y; t < a.T; t += gridDim.y) {
        const type *z = static_cast<const type *>(a.z) + t * a.ldz;
        type *dz = static_cast<type *>(a.dz) + t * a.lddz;
        const int32_t *mask = a.mask ? a.mask + t * a.ldm : nullptr;
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
            if (mask && at < pieces) bits[u] = mask_bits(mask, head + at * VW, VW, a.V);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = base + u * THREADS + (int)threadIdx.x;
            if (at >= pieces) continue;
            float v[VW];
            P::unpack(raw[u], v);
            const int col = head + at * VW;
#pragma unroll
            for (int e = 0; e < VW; ++e) v[e] = row(v[e], bits[u] >> e & 1, col + e);
            P::store(dz + col, v);
        }
        if (VW > 1 && blockIdx.x == gridDim.x - 1 && (int)threadIdx.x < head + a.V - tail0) {
            const int col = (int)threadIdx.x < head ? (int)threadIdx.x : tail0 + (int)threadIdx.x - head;
            const bool allowed = !mask || (mask[col >> 5] >> (col & 31) & 1);
            dz[col] = E::from_float(row(E::to_float(z[col]), allowed, col));
        }
    }
}

}  // namespace sgemm
