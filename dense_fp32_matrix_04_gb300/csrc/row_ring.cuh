// Rows walked by blocks that stay: what the norms and their gradients share.  The
// inputs of the next rows are copied into a ring in shared memory while a row is
// worked on.
#pragma once

#include <cstdint>

#include "ptx.cuh"
#include "rows.cuh"

namespace sgemm {

template <int DT>
__device__ __forceinline__ float load_weight(const void *w, int w_f32, int c) {
    using E = Elem<DT>;
    return w_f32 ? static_cast<const float *>(w)[c] : E::to_float(static_cast<const typename E::type *>(w)[c]);
}

template <int DT>
__device__ __forceinline__ void store_weight(void *w, int w_f32, int64_t c, float v) {
    using E = Elem<DT>;
    if (w_f32) static_cast<float *>(w)[c] = v;
    else static_cast<typename E::type *>(w)[c] = E::from_float(v);
}

// ---------------------------------------------------------------- rows through shared memory
//
// The threads that share a row copy the next rows' inputs into shared memory
// (cp.async, whole 16-byte pieces) while they work on this one, so what is in
// flight does not depend on how many blocks fit an SM.
//
// With ALIGNED rows (16-byte aligned and a whole number of pieces) a warp takes
// NV pieces a lane beside each other, so that one address serves all of them.
// Each thread copies the pieces it will read itself and needs no barrier; its
// pieces past the row's end are copies of nothing, zeros, so that what it reads
// needs no test.  (With a test a piece, and with addresses of their own,
// two thirds of the gradient's instructions were addresses and branches.)
//
// Any other row is copied as the pieces that enclose it (up to 15 bytes in
// front and behind are read and never used), a barrier lets the row's threads
// see each other's copies, and they read single elements, i-th at column
// i * threads + thread.
// 16-byte pieces of the slot of one input of a row, for `threads` threads of `per` elements each
// (the last piece for a row that does not start on one).
__host__ __device__ constexpr int row_pieces(int threads, int per, int size) { return threads * per * size / 16 + 1; }

template <int DT, bool ALIGNED, int NV>
struct RowLayout {
    using type = typename Elem<DT>::type;
    static constexpr int VEC = Elem<DT>::VEC, N = NV * VEC;  // elements a thread
    static constexpr int NEXT = 32 * VEC;                    // columns from a thread's piece to its next
    int D, threads, tx;
    int col, left;  // ALIGNED: this thread's first column, and the columns from there to the row's end

    __device__ explicit RowLayout(int D) : D(D), threads(blockDim.x), tx(threadIdx.x) {
        col = ALIGNED ? ((tx & ~31) * NV + (tx & 31)) * VEC : 0;
        left = D - col;
    }
    // pieces of the slot of one input, and a thread's place in the ring of `rows` slots
    __device__ int pieces() const { return ALIGNED ? NV * 32 : row_pieces(threads, N, sizeof(type)); }
    __device__ uint4 *place(uint4 *ring, int rows) const {
        if constexpr (ALIGNED) {
            const int warp = (threadIdx.y * threads + tx) >> 5;
            return ring + warp * rows * pieces() + (tx & 31);
        } else {
            return ring + threadIdx.y * rows * pieces();
        }
    }
    __device__ bool has(int e) const { return left > e / VEC * NEXT; }  // ALIGNED: the piece of element e
    __device__ static int at(int e) { return e / VEC * NEXT + e % VEC; }
    // The functions below take rows from this thread's first column (ALIGNED) or their start, and
    // slots from this thread's place.
    __device__ void copy(uint4 *slot, const type *row) const {
        if constexpr (ALIGNED) {
#pragma unroll
            for (int v = 0; v < NV; ++v)
                cp_async_16(smem_addr(slot + v * 32), row + v * NEXT, has(v * VEC) ? 16 : 0);
        } else {
            const uintptr_t lo = reinterpret_cast<uintptr_t>(row) & ~(uintptr_t)15;
            const int n = (int)((reinterpret_cast<uintptr_t>(row + D) + 15 - lo) >> 4);
            for (int p = tx; p < n; p += threads)
                cp_async_16(smem_addr(slot + p), reinterpret_cast<const void *>(lo + 16 * (uintptr_t)p), 16);
        }
    }
    template <int COUNT>
    __device__ static void unpack(const type *p, F2 (&out)[COUNT / 2]) {
        float f[8];
        if constexpr (sizeof(type) * COUNT == 16) {
            unpack16<DT>(*reinterpret_cast<const uint4 *>(p), f);
        } else {
            const uint2 w = *reinterpret_cast<const uint2 *>(p);
            unpack16<DT>(make_uint4(w.x, w.y, 0, 0), f);
        }
#pragma unroll
        for (int i = 0; i < COUNT / 2; ++i) out[i] = F2(f[2 * i], f[2 * i + 1]);
    }
    // COUNT elements (a piece, or four of one) from this thread's e-th of the row that was copied
    // from `row`; 0 past its end
    template <int COUNT>
    __device__ void read(const uint4 *slot, const type *row, int e, F2 (&out)[COUNT / 2]) const {
        if constexpr (ALIGNED) {
            unpack<COUNT>(reinterpret_cast<const type *>(slot + e / VEC * 32) + e % VEC, out);
        } else {
            const type *q = reinterpret_cast<const type *>(slot) + (reinterpret_cast<uintptr_t>(row) & 15) / sizeof(type);
            auto one = [&](int i) { return i * threads + tx < D ? Elem<DT>::to_float(q[i * threads + tx]) : 0.f; };
#pragma unroll
            for (int i = 0; i < COUNT; i += 2) out[i / 2] = F2(one(e + i), one(e + i + 1));
        }
    }
    // the same of weights (from the block's first column); ALIGNED weights start on 16 bytes.
    // FOR_ZEROS: they meet only zeros past the row's end, and are the row's last ones there.
    template <int COUNT, bool FOR_ZEROS = false>
    __device__ void weights(const void *w, int w_f32, int e, F2 (&out)[COUNT / 2]) const {
        if constexpr (ALIGNED && FOR_ZEROS) {
            const int c = (has(e) ? col + e / VEC * NEXT : D - VEC) + e % VEC;
            if (w_f32) {
#pragma unroll
                for (int i = 0; i < COUNT; i += 4) {
                    const float4 f = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(w) + c + i));
                    out[i / 2] = F2(f.x, f.y), out[i / 2 + 1] = F2(f.z, f.w);
                }
            } else {
                unpack<COUNT>(static_cast<const type *>(w) + c, out);
            }
        } else if constexpr (ALIGNED) {
#pragma unroll
            for (int i = 0; i < COUNT / 2; ++i) out[i] = F2(0.f);
            if (w_f32) {
#pragma unroll
                for (int i = 0; i < COUNT; i += 4)
                    if (has(e)) {
                        const float4 f = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(w) + col + at(e + i)));
                        out[i / 2] = F2(f.x, f.y), out[i / 2 + 1] = F2(f.z, f.w);
                    }
            } else if (has(e)) {
                unpack<COUNT>(static_cast<const type *>(w) + col + at(e), out);
            }
        } else {
            auto one = [&](int i) { return i * threads + tx < D ? load_weight<DT>(w, w_f32, i * threads + tx) : 0.f; };
#pragma unroll
            for (int i = 0; i < COUNT; i += 2) out[i / 2] = F2(one(e + i), one(e + i + 1));
        }
    }
    // a piece from this thread's e-th element on
    __device__ void store(type *row, int e, const F2 *v) const {
        float f[VEC];
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
            const float2 b = v[i].both();
            f[2 * i] = b.x;
            f[2 * i + 1] = b.y;
        }
        if constexpr (ALIGNED) {
            if (has(e)) *reinterpret_cast<uint4 *>(row + at(e)) = pack16<DT>(f);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if ((e + i) * threads + tx < D) row[(e + i) * threads + tx] = Elem<DT>::from_float(f[i]);
        }
    }
    // a piece's values as `store` rounds them
    __device__ static void rounded(F2 *v) {
        if constexpr (DT != SGEMM_F32) {
            float f[VEC];
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) {
                const float2 b = v[i].both();
                f[2 * i] = b.x;
                f[2 * i + 1] = b.y;
            }
            unpack16<DT>(pack16<DT>(f), f);
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) v[i] = F2(f[2 * i], f[2 * i + 1]);
        }
    }
    // 0 in the place of the elements e and e + 1 where they lie past the row's end
    __device__ void only_inside(int e, F2 &d) const {
        if constexpr (ALIGNED) {
            if (!has(e)) d = F2(0.f);
        } else {
            const float2 f = d.both();
            d = F2(e * threads + tx < D ? f.x : 0.f, (e + 1) * threads + tx < D ? f.y : 0.f);
        }
    }
    // how many columns this thread's warp has
    __device__ float warp_columns() const {
        if constexpr (ALIGNED) return (float)min(max(D - (tx >> 5) * NV * NEXT, 0), NV * NEXT);
        int n = 0;
        for (int i = 0; i < N; ++i) n += min(max(D - i * threads - (tx & ~31), 0), 32);
        return (float)n;
    }
    // stores FP32 sums, four columns at a time where a thread has them beside each other
    // (single floats would write every sector eight times)
    __device__ void put(float *row, int e, const F2 *v, bool add) const {
        if constexpr (ALIGNED) {
            if (has(e))
#pragma unroll
                for (int i = 0; i < VEC / 2; i += 2) {
                    float4 *p = reinterpret_cast<float4 *>(row + at(e + 2 * i));
                    const float2 f = v[i].both(), g = v[i + 1].both();
                    float4 s = make_float4(f.x, f.y, g.x, g.y);
                    if (add) {
                        const float4 o = *p;
                        s = make_float4(o.x + s.x, o.y + s.y, o.z + s.z, o.w + s.w);
                    }
                    *p = s;
                }
        } else {
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) {
                const float2 f = v[i].both();
                const int c = (e + 2 * i) * threads + tx, c1 = c + threads;
                if (c < D) row[c] = add ? row[c] + f.x : f.x;
                if (c1 < D) row[c1] = add ? row[c1] + f.y : f.y;
            }
        }
    }
};

// The barrier of the threads that share a row.
__device__ __forceinline__ void row_sync(int warps) {
    if (warps == 1) __syncwarp();
    else __syncthreads();
}

// Runner b (a block, or a warp of one) takes consecutive rows, so that a gate
// row's sum stays in registers until the row changes: T / runners of them, and
// the first T % runners runners one more.  No division of 64 bits is on the way
// of a row (each cost about 100 instructions).
struct RowRuns {
    int each, more;
    __device__ RowRuns(int T, int runners) : each(T / runners), more(T % runners) {}
    __device__ int first(int b) const { return b * each + min(b, more); }
    __device__ int runner_of(int t) const {
        const int wide = more * (each + 1);
        return t < wide ? t / (each + 1) : more + (t - wide) / each;
    }
};

}  // namespace sgemm
