// row8.cuh -- a row of a matrix held by a group of threads, V times eight
// elements each, as fp32 (the operators that need a whole row at once), and
// sums over the group.
//
// How rows are moved (Access):
//   kVec      the thread's eight are neighbours, moved 16 (bf16) or 32 bytes (fp32) at
//     a time; rows start on 16 bytes and the columns are a multiple of 8.
//   kStrided  rows start anywhere; the eight lie `tpr` columns apart and go one by one, a
//     warp's together in whole lines.
//   kShifted  rows start anywhere; the eight are neighbours.  A thread loads the aligned
//     16-byte pieces that they lie in, as far as those lie inside the row, and shifts; it
//     stores the aligned pieces that begin in them, the last with its neighbour's
//     first elements.  At the ends of the row (and of the warp, for stores) elements go
//     one by one.
//     Groups are whole warps.
// Strided against shifted, us, bf16: combination of 2000 x 2047 with 6 choices 60 / 36,
// quantisation of 4096 x 4095 16.6 / 11.3; but residual_norm of 16384 x 4095 264 / 308 and
// its gradients of 4096 x 2047 84 / 100, which instructions bound already.
#pragma once
#include "activation.cuh"
#include "gbr_ptx.cuh"
#include "vec8.cuh"

namespace gbr {

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f32(float x, float* y) { *y = x; }
__device__ __forceinline__ void from_f32(float x, __nv_bfloat16* y) { *y = __float2bfloat16_rn(x); }

enum Access : int { kStrided = 0, kVec = 1, kShifted = 2 };

// First column of vector v of thread `t` of `tpr`, of neighbours; column of element j, strided.
__device__ __forceinline__ int32_t row_col(int v, int32_t t, int32_t tpr) { return (v * tpr + t) * 8; }
__device__ __forceinline__ int32_t strided_col(int v, int j, int32_t t, int32_t tpr) { return (v * 8 + j) * tpr + t; }

// Eight elements as they are loaded; columns past the end are zero.
template <typename T>
struct Raw8 {
    uint32_t w[sizeof(T) * 2];
};

// Elements from the aligned address in front of an element to that element.
__device__ __forceinline__ int32_t off_16(const __nv_bfloat16* p) { return int32_t(reinterpret_cast<uintptr_t>(p) / 2 % 8); }
__device__ __forceinline__ int32_t off_16(const float* p) { return int32_t(reinterpret_cast<uintptr_t>(p) / 4 % 4); }

// out = eight elements of `w` from element `by` on (below 8 of bf16, 4 of fp32).
__device__ __forceinline__ void shift8(Raw8<__nv_bfloat16>& out, const uint32_t (&w)[8], int32_t by) {
    uint32_t x[7];
    const bool four = by & 4, two = by & 2, one = by & 1;
#pragma unroll
    for (int i = 0; i < 7; ++i) x[i] = four ? (i + 2 < 8 ? w[i + 2] : 0u) : w[i];
#pragma unroll
    for (int i = 0; i < 6; ++i) x[i] = two ? x[i + 1] : x[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) out.w[i] = one ? __funnelshift_r(x[i], x[i + 1], 16) : x[i];
}
__device__ __forceinline__ void shift8(Raw8<float>& out, const uint32_t (&w)[12], int32_t by) {
    uint32_t x[10];
    const bool two = by & 2, one = by & 1;
#pragma unroll
    for (int i = 0; i < 10; ++i) x[i] = two ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 8; ++i) out.w[i] = one ? x[i + 1] : x[i];
}

__device__ __forceinline__ void take_piece(uint32_t* w, const uint4& x) { w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w; }

template <int A>
__device__ __forceinline__ void load_raw8(Raw8<__nv_bfloat16>& r, const __nv_bfloat16* row, int v, int32_t t,
                                          int32_t tpr, int32_t cols) {
    const int32_t c = row_col(v, t, tpr), left = cols - c;
    uint4 x = make_uint4(0, 0, 0, 0);
    if (A == kVec) {
        if (left > 0) x = *reinterpret_cast<const uint4*>(row + c);
        take_piece(r.w, x);
        return;
    }
    if (A == kStrided) {
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const int32_t d = strided_col(v, j, t, tpr), e = d + tpr;
            const uint32_t lo = d < cols ? __bfloat16_as_ushort(row[d]) : 0u;
            const uint32_t hi = e < cols ? __bfloat16_as_ushort(row[e]) : 0u;
            r.w[j / 2] = lo | (hi << 16);
        }
        return;
    }
    const int32_t off = off_16(row + c);
    // Inside the row: from `off` elements before the first (c is a multiple of 8) to 8 after those.
    if (off == 0 ? left >= 8 : c > 0 && left >= 16 - off) {
        const uint4* p = reinterpret_cast<const uint4*>(row + c - off);
        uint32_t w[8];
        take_piece(w, p[0]);
        take_piece(w + 4, off == 0 ? x : p[1]);
        shift8(r, w, off);
    } else {
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const uint32_t lo = j < left ? __bfloat16_as_ushort(row[c + j]) : 0u;
            const uint32_t hi = j + 1 < left ? __bfloat16_as_ushort(row[c + j + 1]) : 0u;
            r.w[j / 2] = lo | (hi << 16);
        }
    }
}
template <int A>
__device__ __forceinline__ void load_raw8(Raw8<float>& r, const float* row, int v, int32_t t, int32_t tpr, int32_t cols) {
    const int32_t c = row_col(v, t, tpr), left = cols - c;
    uint4 x = make_uint4(0, 0, 0, 0), y = x;
    if (A == kVec) {
        if (left > 0) {
            x = reinterpret_cast<const uint4*>(row + c)[0];
            y = reinterpret_cast<const uint4*>(row + c)[1];
        }
        take_piece(r.w, x), take_piece(r.w + 4, y);
        return;
    }
    if (A == kStrided) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int32_t d = strided_col(v, j, t, tpr);
            r.w[j] = d < cols ? __float_as_uint(row[d]) : 0u;
        }
        return;
    }
    const int32_t off = off_16(row + c);
    if (off == 0 ? left >= 8 : c > 0 && left >= 12 - off) {
        const uint4* p = reinterpret_cast<const uint4*>(row + c - off);
        uint32_t w[12];
        take_piece(w, p[0]), take_piece(w + 4, p[1]);
        take_piece(w + 8, off == 0 ? x : p[2]);
        shift8(r, w, off);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) r.w[j] = j < left ? __float_as_uint(row[c + j]) : 0u;
    }
}

__device__ __forceinline__ float raw_at(const Raw8<__nv_bfloat16>& r, int j) {
    return __uint_as_float(j % 2 ? r.w[j / 2] & 0xFFFF0000u : r.w[j / 2] << 16);
}
__device__ __forceinline__ float raw_at(const Raw8<float>& r, int j) { return __uint_as_float(r.w[j]); }

template <typename T, int A>
__device__ __forceinline__ void load_row8(float (&x)[8], const T* row, int v, int32_t t, int32_t tpr, int32_t cols) {
    Raw8<T> r;
    load_raw8<A>(r, row, v, t, tpr, cols);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = raw_at(r, j);
}

// Shifted, every lane of a warp calls the stores, those without columns too.
template <int A>
__device__ __forceinline__ void store_raw8(__nv_bfloat16* row, const Raw8<__nv_bfloat16>& r, int v, int32_t t, int32_t tpr,
                                           int32_t cols) {
    const int32_t c = row_col(v, t, tpr), left = cols - c;
    if (A == kVec) {
        if (left > 0) *reinterpret_cast<uint4*>(row + c) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
        return;
    }
    if (A == kStrided) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int32_t d = strided_col(v, j, t, tpr);
            if (d < cols) row[d] = __ushort_as_bfloat16(uint16_t(j % 2 ? r.w[j / 2] >> 16 : r.w[j / 2] & 0xFFFFu));
        }
        return;
    }
    const int32_t off = off_16(row + c), lane = t % 32;
    uint32_t w[8];                                      // this thread's and the next one's
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[i] = r.w[i];
        w[4 + i] = __shfl_down_sync(0xffffffffu, r.w[i], 1);
    }
    // The aligned piece that begins in this thread's elements, whole inside the row and with a neighbour for its rest;
    // the piece in front of it is the last thread's, under the same conditions.
    const int32_t from = (8 - off) % 8;
    const bool piece = off == 0 ? left >= 8 : lane < 31 && left >= 16 - off;
    const bool front = off != 0 && lane > 0 && left >= 8 - off;
    if (piece) {
        Raw8<__nv_bfloat16> x;
        shift8(x, w, from);
        *reinterpret_cast<uint4*>(row + c + from) = make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]);
    }
    if (piece && (front || off == 0)) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (j >= left || (j < from ? front : piece)) continue;
        row[c + j] = __ushort_as_bfloat16(uint16_t(j % 2 ? r.w[j / 2] >> 16 : r.w[j / 2] & 0xFFFFu));
    }
}
template <int A>
__device__ __forceinline__ void store_raw8(float* row, const Raw8<float>& r, int v, int32_t t, int32_t tpr, int32_t cols) {
    const int32_t c = row_col(v, t, tpr), left = cols - c;
    if (A == kVec) {
        if (left <= 0) return;
        reinterpret_cast<uint4*>(row + c)[0] = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
        reinterpret_cast<uint4*>(row + c)[1] = make_uint4(r.w[4], r.w[5], r.w[6], r.w[7]);
        return;
    }
    if (A == kStrided) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int32_t d = strided_col(v, j, t, tpr);
            if (d < cols) row[d] = __uint_as_float(r.w[j]);
        }
        return;
    }
    const int32_t off = off_16(row + c), lane = t % 32;
    uint32_t w[12];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = r.w[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[8 + i] = __shfl_down_sync(0xffffffffu, r.w[i], 1);
    // Two aligned pieces begin in this thread's elements; the first needs no neighbour.
    const int32_t from = (4 - off) % 4;
    const bool first = left >= from + 4, second = off == 0 ? left >= 8 : lane < 31 && left >= 12 - off;
    const bool front = off != 0 && lane > 0 && left >= 4 - off;
    Raw8<float> x;
    shift8(x, w, from);
    if (first) *reinterpret_cast<uint4*>(row + c + from) = make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]);
    if (second) *reinterpret_cast<uint4*>(row + c + from + 4) = make_uint4(x.w[4], x.w[5], x.w[6], x.w[7]);
    if (second && (front || off == 0)) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (j >= left || (j < from ? front : j < from + 4 ? first : second)) continue;
        row[c + j] = __uint_as_float(r.w[j]);
    }
}

// Rounded to the type.
__device__ __forceinline__ void round8(Raw8<__nv_bfloat16>& r, const float (&x)[8]) { take_piece(r.w, pack8(x)); }
__device__ __forceinline__ void round8(Raw8<float>& r, const float (&x)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) r.w[j] = __float_as_uint(x[j]);
}

template <typename T, int A>
__device__ __forceinline__ void store_row8(T* row, const float (&x)[8], int v, int32_t t, int32_t tpr, int32_t cols) {
    Raw8<T> r;
    round8(r, x);
    store_raw8<A>(row, r, v, t, tpr, cols);
}

// The same as four pairs, which one instruction multiplies or adds (activation.cuh).
__device__ __forceinline__ F2 raw_pair(const Raw8<__nv_bfloat16>& r, int i) {
    return f2(__uint_as_float(r.w[i] << 16), __uint_as_float(r.w[i] & 0xFFFF0000u));
}
__device__ __forceinline__ F2 raw_pair(const Raw8<float>& r, int i) {
    return f2(__uint_as_float(r.w[2 * i]), __uint_as_float(r.w[2 * i + 1]));
}
__device__ __forceinline__ float sum_pair(F2 x) {
    float a, b;
    split2(x, a, b);
    return a + b;
}
template <typename T, int A>
__device__ __forceinline__ void load_pairs(F2 (&x)[4], const T* row, int v, int32_t t, int32_t tpr, int32_t cols) {
    Raw8<T> r;
    load_raw8<A>(r, row, v, t, tpr, cols);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = raw_pair(r, i);
}
template <typename T, int A>
__device__ __forceinline__ void store_pairs(T* row, const F2 (&x)[4], int v, int32_t t, int32_t tpr, int32_t cols) {
    float y[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) split2(x[i], y[2 * i], y[2 * i + 1]);
    store_row8<T, A>(row, y, v, t, tpr, cols);
}

// Four pairs of a thread in shared memory: two pieces of 16 bytes, each next to its neighbours'.
__device__ __forceinline__ void put_pairs(uint32_t at, const F2 (&x)[4]) {
    float y[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) split2(x[i], y[2 * i], y[2 * i + 1]);
#pragma unroll
    for (int h = 0; h < 2; ++h)
        ptx::st_shared_v4(at + uint32_t(h) * 16u * blockDim.x, __float_as_uint(y[4 * h]), __float_as_uint(y[4 * h + 1]),
                          __float_as_uint(y[4 * h + 2]), __float_as_uint(y[4 * h + 3]));
}
__device__ __forceinline__ void get_pairs(F2 (&x)[4], uint32_t at) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint4 w = ptx::ld_shared_v4(at + uint32_t(h) * 16u * blockDim.x);
        x[2 * h] = f2(__uint_as_float(w.x), __uint_as_float(w.y));
        x[2 * h + 1] = f2(__uint_as_float(w.z), __uint_as_float(w.w));
    }
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int d = 16; d > 0; d /= 2) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

// Sums of N (1 to 4) values over groups of `tpr` threads, whole warps or, for one value, a power of two below 32; this
// thread's is `group`.  Every
// thread of the block calls it; `buf` is this call's own until the next __syncthreads.  The order of the sum is fixed.
//
// Several values take the shuffles of little more than one: after the first step each half of the warp goes on with two
// of four, after the second each quarter with one, whose lanes also join the warps' sums.  (Shuffles and what goes with
// them bound the gradients' rows: 4096 columns on 16 warps, three sums and one, took 50 shuffles a warp and row one value
// at a time, 20 this way.)
__device__ __forceinline__ float fold4(float x0, float x1, float x2, float x3, int32_t lane) {
    const bool upper = lane & 16, odd = lane & 8;
    float a = upper ? x2 : x0, b = upper ? x3 : x1;
    a += __shfl_xor_sync(0xffffffffu, upper ? x0 : x2, 16);
    b += __shfl_xor_sync(0xffffffffu, upper ? x1 : x3, 16);
    float c = odd ? b : a;
    c += __shfl_xor_sync(0xffffffffu, odd ? a : b, 8);
#pragma unroll
    for (int d = 4; d > 0; d /= 2) c += __shfl_xor_sync(0xffffffffu, c, d);
    return c;                                           // of value lane / 8
}

template <int N>
__device__ __forceinline__ void group_sum(float (&x)[N], float (*buf)[32], int32_t tpr, int32_t group) {
    if (N == 1 && tpr < 32) {                           // several groups a warp
        for (int d = tpr / 2; d > 0; d /= 2) x[0] += __shfl_xor_sync(0xffffffffu, x[0], d);
        return;
    }
    const int32_t lane = int32_t(threadIdx.x) % 32, warp = int32_t(threadIdx.x) / 32, warps = tpr / 32;
    const int32_t first = group * warps;
    if (N == 1) {
        x[0] = warp_sum(x[0]);
        if (tpr == 32) return;
        if (lane == 0) buf[0][warp] = x[0];
        __syncthreads();
        x[0] = warp_sum(lane < warps ? buf[0][first + lane] : 0.f);
        return;
    }
    float c = fold4(x[0], x[N > 1 ? 1 : 0], N > 2 ? x[N > 2 ? 2 : 0] : 0.f, N > 3 ? x[N > 3 ? 3 : 0] : 0.f, lane);
    if (tpr > 32) {
        const int32_t value = lane / 8, l = lane % 8;
        if (l == 0 && value < N) buf[value][warp] = c;
        __syncthreads();
        c = 0.f;
        if (value < N)
#pragma unroll
            for (int w = 0; w < 32; w += 8)
                if (w + l < warps) c += buf[value][first + w + l];
#pragma unroll
        for (int d = 4; d > 0; d /= 2) c += __shfl_xor_sync(0xffffffffu, c, d);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = __shfl_sync(0xffffffffu, c, 8 * i);
}

// A row cut over the `parts` (at most 4) CTAs of a cluster: x, each CTA's sums, become the cluster's, added in rank order.
// Every thread of the cluster calls it; `slot` is this and the next call's in turn (a CTA writes the next call's when
// others may still read this one's, but the one after only when all have come to the next).
template <int N>
__device__ __forceinline__ void cluster_sum(float (&x)[N], float (*slot)[4], uint32_t parts, uint32_t rank) {
    static_assert(N <= 4);
    if (threadIdx.x < parts) {
        const uint32_t to = ptx::mapa_shared(ptx::smem_addr(&slot[rank][0]), threadIdx.x);
#pragma unroll
        for (int i = 0; i < N; ++i) ptx::st_shared_cluster_u32(to + 4u * uint32_t(i), __float_as_uint(x[i]));
    }
    ptx::cluster_sync_all();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        x[i] = slot[0][i];
#pragma unroll
        for (uint32_t r = 1; r < 4; ++r)
            if (r < parts) x[i] += slot[r][i];
    }
}

// Asynchronous copies of a thread's own 16-byte pieces, group by group.
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Vector v of a row into shared memory, where the row lies as it is, and from there.
template <typename T>
__device__ __forceinline__ void copy_row8(uint32_t to, const T* row, int v, int32_t t, int32_t tpr, int32_t cols) {
    const int32_t c = row_col(v, t, tpr);
    if (c >= cols) return;
#pragma unroll
    for (int i = 0; i < int(sizeof(T) / 2); ++i)
        ptx::cp_async_16(to + uint32_t(c) * uint32_t(sizeof(T)) + 16u * i, reinterpret_cast<const uint8_t*>(row + c) + 16 * i, 16);
}
// (What lies past the last column has to be zero there.)
template <typename T>
__device__ __forceinline__ void take_row8(Raw8<T>& r, uint32_t from, int v, int32_t t, int32_t tpr) {
    const uint32_t at = from + uint32_t(row_col(v, t, tpr)) * uint32_t(sizeof(T));
#pragma unroll
    for (int i = 0; i < int(sizeof(T) / 2); ++i) {
        const uint4 x = ptx::ld_shared_v4(at + 16u * i);
        r.w[4 * i] = x.x, r.w[4 * i + 1] = x.y, r.w[4 * i + 2] = x.z, r.w[4 * i + 3] = x.w;
    }
}
// Zeroes a thread's places of `rows` rows of `row_bytes` past the last column.
template <typename T, int V>
__device__ __forceinline__ void clear_past(uint32_t ring, uint32_t rows, uint32_t row_bytes, int32_t t, int32_t tpr,
                                           int32_t cols) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int32_t c = row_col(v, t, tpr);
        if (c < cols) continue;
        for (uint32_t r = 0; r < rows; ++r)
#pragma unroll
            for (int i = 0; i < int(sizeof(T) / 2); ++i)
                ptx::st_shared_v4(ring + r * row_bytes + uint32_t(c) * uint32_t(sizeof(T)) + 16u * i, 0, 0, 0, 0);
    }
}

// Rows that start anywhere but whose operands all start alike: a row from the aligned address in front of it, `off`
// elements before its first.  Columns are counted from there, up to `end`; those in front of the row become zero.
template <typename T>
__device__ __forceinline__ void copy_row8_from(uint32_t to, const T* at, int v, int32_t t, int32_t tpr, int32_t end) {
    constexpr int32_t kPiece = 16 / int32_t(sizeof(T));
    const int32_t c = row_col(v, t, tpr);
    if (c >= end) return;
#pragma unroll
    for (int i = 0; i < int(sizeof(T) / 2); ++i) {
        const int32_t e = c + i * kPiece, n = end - e < kPiece ? end - e : kPiece;
        ptx::cp_async_16(to + uint32_t(e) * uint32_t(sizeof(T)), at + (n > 0 ? e : c), n > 0 ? uint32_t(n) * uint32_t(sizeof(T)) : 0u);
    }
}
__device__ __forceinline__ void clear_front(Raw8<__nv_bfloat16>& r, int32_t off) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < off) r.w[j / 2] &= j % 2 ? 0x0000FFFFu : 0xFFFF0000u;
}
__device__ __forceinline__ void clear_front(Raw8<float>& r, int32_t off) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (j < off) r.w[j] = 0u;
}
template <typename T>
__device__ __forceinline__ void load_pairs_from(F2 (&x)[4], const T* row, int v, int32_t t, int32_t tpr, int32_t off,
                                                int32_t end) {
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int32_t c = row_col(v, t, tpr) + j;
        y[j] = c >= off && c < end ? to_f32(row[c - off]) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = f2(y[2 * i], y[2 * i + 1]);
}
// `at` is the aligned address; element by element where `each`, at row - off, which need not be aligned then.
template <typename T>
__device__ __forceinline__ void store_pairs_from(T* at, const F2 (&x)[4], int v, int32_t t, int32_t tpr, int32_t off,
                                                 int32_t end, bool each = false) {
    const int32_t c = row_col(v, t, tpr);
    if (!each && c >= off && c + 8 <= end) {
        store_pairs<T, kVec>(at, x, v, t, tpr, end);
        return;
    }
    float y[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) split2(x[i], y[2 * i], y[2 * i + 1]);
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (c + j >= off && c + j < end) from_f32(y[j], at + c + j);
}

}  // namespace gbr
