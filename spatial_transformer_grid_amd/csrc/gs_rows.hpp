// gs_rows.hpp -- rows of a matrix in the registers of the threads that share
// them: loads, stores and sums over a row, for the operators that normalise.
#pragma once

#include "gs_tokens.hpp"

namespace gs {

template <int N>
__device__ __forceinline__ float lanes_total(float v) {
#pragma unroll
    for (int s = 1; s < N; s <<= 1) v += __shfl_xor(v, s);
    return v;
}

// The same sums, bit for bit, without a way through LDS: neighbours, pairs, halves
// of eight and of sixteen lanes by the lane permutations of an addition (a mirrored
// lane's partial sum is that of the lane across), then halves of 32 and of the wave.
template <int CTRL>
__device__ __forceinline__ float plus_lane(float v) {
    return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}

template <int N>
__device__ __forceinline__ float lanes_sum(float v) {
    static_assert(N == 8 || N == 32 || N == 64, "widths of a row's lanes");
    v = plus_lane<0xB1>(v);                          // quad_perm [1, 0, 3, 2]
    v = plus_lane<0x4E>(v);                          // quad_perm [2, 3, 0, 1]
    v = plus_lane<0x141>(v);                         // row_half_mirror
    if constexpr (N > 8) {
        v = plus_lane<0x140>(v);                     // row_mirror
        const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v),
                                                        false, false);
        v = __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
    }
    if constexpr (N > 32) v += other_half(v);
    return v;
}

// Sums over the NT threads of a row, two at once; `red` holds 2 NT / 64 floats
// where they are more than a wave.
template <int NT>
__device__ __forceinline__ void row_totals(float &a, float &b, float *red) {
    a = lanes_total<(NT < 64 ? NT : 64)>(a);
    b = lanes_total<(NT < 64 ? NT : 64)>(b);
    if constexpr (NT > 64) {
        constexpr int W = NT / 64;
        __syncthreads();
        if ((threadIdx.x & 63) == 0) {
            red[threadIdx.x >> 6] = a;
            red[W + (threadIdx.x >> 6)] = b;
        }
        __syncthreads();
        a = b = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            a += red[w];
            b += red[W + w];
        }
    }
}

template <int NT>
__device__ __forceinline__ float row_total(float v, float *red) {
    float none = 0.0f;
    row_totals<NT>(v, none, red);
    return v;
}

template <typename T>
__device__ __forceinline__ float param(const void *v, int64_t i, int f32) {
    if (f32) return ((const float *)v)[i];
    return T::from_raw(((const typename T::raw_t *)v)[i]);
}

// A thread's E elements of a row: eight neighbours of every chunk t + NT j where
// rows allow 16-byte accesses (VEC), else the elements t + NT j.
template <int NT, bool VEC>
__device__ __forceinline__ int column(int t, int e) {
    return VEC ? 8 * (t + NT * (e >> 3)) + (e & 7) : t + NT * e;
}

template <typename T, int NT, int E, bool VEC>
__device__ __forceinline__ void load_row(const typename T::raw_t *row, int cols, int t, float *v) {
    if constexpr (VEC) {
#pragma unroll
        for (int e = 0; e < E; e += 8) {
            const int c = column<NT, true>(t, e);
            const Frag<T> f = frag_global<T>(row, c, cols, c < cols, true);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[e + j] = frag_get<T>(f, j);
        }
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int c = column<NT, false>(t, e);
            v[e] = c < cols ? T::from_raw(row[c]) : 0.0f;
        }
    }
}

template <typename T, int NT, int E, bool VEC>
__device__ __forceinline__ void store_row(typename T::raw_t *row, int cols, int t, const float *v) {
    if constexpr (VEC) {
#pragma unroll
        for (int e = 0; e < E; e += 8) {
            const int c = column<NT, true>(t, e);
            const Frag<T> f = frag_pack<T>(v + e);
            if (c < cols)
#pragma unroll
                for (int i = 0; i < T::bytes / 2; ++i) *(u32x4 *)(row + c + i * (16 / T::bytes)) = f.w[i];
        }
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int c = column<NT, false>(t, e);
            if (c < cols) row[c] = to_bits<T>(v[e]);
        }
    }
}

template <typename T, int NT, int E, bool VEC>
__device__ __forceinline__ void load_params(const void *src, int f32, int cols, int t, float *v) {
    if (!src) {
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = 0.0f;
    } else if (f32) {
        load_row<F32, NT, E, VEC>((const uint32_t *)src, cols, t, v);
    } else {
        load_row<T, NT, E, VEC>((const typename T::raw_t *)src, cols, t, v);
    }
}

}  // namespace gs
