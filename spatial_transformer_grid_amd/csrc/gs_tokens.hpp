// gs_tokens.hpp -- shared parts of the token operators (layer norm, dropout,
// attention): launch parameters, the counter-based generator, 8-element
// fragments of the matrix cores.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gs {

constexpr int kMaxBuckets = 512;     // buckets of a bias table
constexpr int kMaxBorder = 1024;     // largest first distance of a last bucket

struct NormParams {
    const void *X, *dY, *scale, *bias;
    void *Y, *dX;
    float *mean, *inv_std;
    int64_t rows;
    int cols;
    int64_t x_stride, y_stride, dy_stride, dx_stride;
    float epsilon;
    int param_f32;            // scale and bias are fp32 (else the data type)
    int vec;                  // rows allow 16-byte accesses
    void *dscale, *dbias;
    float *partial;           // backward: (parts, 2, cols) sums
    int parts;
};

struct DropoutParams {
    const void *X, *residual;
    void *Y;
    int64_t count;
    uint32_t threshold, seed_lo, seed_hi, call;
    float keep_scale;
    int vec;
};

struct AttnParams {
    const void *q, *k, *v, *o_in, *d_o, *table;
    void *o, *dq, *dk, *dv, *dtable;
    float *lse;
    const int32_t *lengths;
    float *delta;             // backward: (B, H, Lq) row sums of dO * O
    float *part;              // backward: (H, B * q_tiles, buckets) sums of dS
    float *split;             // forward, split keys: partial O, then (max, sum)
    int64_t qs[3], ks[3], vs[3], os[3], dos[3], dqs[3], dks[3], dvs[3];
    int B, H, Hkv, G, Lq, Lk, D;
    int causal, from_end, first;
    float scale, scale2;      // scale2 = scale * log2(e)
    int buckets, side, border, bidirectional, table_f32;
    int lut;                  // entries of the distance table (0: no bias)
    uint32_t threshold, seed_lo, seed_hi, call;
    float keep_scale;
    int vec;                  // rows of every tensor allow 16-byte accesses
    int tiles;                // query tiles (key tiles in the dK / dV kernel)
    int splits;               // forward, few queries: parts of the key axis
    int nblocks;
    uint16_t starts[kMaxBuckets];  // first distance of each bucket of one side
};

// Launchers; 0 or the hipError_t of the launch.  `dtype` 0 f32, 1 f16, 2 bf16.
int launch_layer_norm(const NormParams &p, int dtype, hipStream_t stream);
int launch_layer_norm_backward(const NormParams &p, int dtype, hipStream_t stream);
int layer_norm_parts(int64_t rows, int64_t cols);
int launch_dropout(const DropoutParams &p, int dtype, hipStream_t stream);
int launch_attention(const AttnParams &p, int dtype, hipStream_t stream);
int launch_attention_backward(const AttnParams &p, int dtype, hipStream_t stream);

constexpr int kAttnQueries = 128;    // queries of a block, keys of a dK / dV block

}  // namespace gs

#if defined(__HIPCC__)
#include "gs_device.hpp"

namespace gs {

typedef __attribute__((ext_vector_type(4))) float tokens_f32x4;
typedef __attribute__((ext_vector_type(2))) unsigned int u32x2;
typedef __attribute__((ext_vector_type(16))) float f32x16;
typedef __bf16 bf16v8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16v8 __attribute__((ext_vector_type(8)));
typedef short s16v4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// fp32 -> the raw bits of T, to nearest even
template <typename T>
__device__ __forceinline__ typename T::raw_t to_bits(float v) {
    if constexpr (T::bytes == 4) return __builtin_bit_cast(uint32_t, v);
    else if constexpr (__is_same(T, BF16)) return __builtin_bit_cast(uint16_t, (__bf16)settle(v));
    else return __builtin_bit_cast(uint16_t, (_Float16)settle(v));
}

// Philox4x32-10 (Salmon, Moraes, Dror, Shaw 2011): ten rounds of two 32 x 32
// -> 64-bit products each.  What bounds it is the rate of the 32-bit integer
// multiplier, a quarter of the vector rate; one call serves eight elements.
__device__ __forceinline__ u32x4 philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3,
                                        uint32_t k0, uint32_t k1) {
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
        const uint32_t n0 = (uint32_t)(b >> 32) ^ c1 ^ k0, n2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
        c1 = (uint32_t)b;
        c3 = (uint32_t)a;
        c0 = n0;
        c2 = n2;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return u32x4{c0, c1, c2, c3};
}

// Number e (0..7) of a call: low half of the first word first.
__device__ __forceinline__ bool kept(const u32x4 &r, int e, uint32_t threshold) {
    const uint32_t w = r[e >> 1];
    return ((e & 1) ? w >> 16 : w & 0xffffu) >= threshold;
}

// Eight consecutive elements of T along the contracted axis: what a lane
// feeds the 32 x 32 matrix instructions for 16 steps of that axis (lanes 0-31
// the first eight, lanes 32-63 the last eight).
template <typename T>
struct Frag {
    u32x4 w[T::bytes / 2];
};

template <typename T>
__device__ __forceinline__ float frag_get(const Frag<T> &f, int j) {
    if constexpr (T::bytes == 4) return __builtin_bit_cast(float, (uint32_t)f.w[j >> 2][j & 3]);
    else return T::from_raw((uint16_t)(f.w[0][j >> 1] >> (16 * (j & 1))));
}

template <typename T>
__device__ __forceinline__ Frag<T> frag_pack(const float *v) {
    Frag<T> f;
    if constexpr (T::bytes == 4) {
#pragma unroll
        for (int j = 0; j < 8; ++j) f.w[j >> 2][j & 3] = __builtin_bit_cast(uint32_t, v[j]);
    } else if constexpr (__is_same(T, BF16)) {
        bf16v8 x;
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = (__bf16)v[j];
        f.w[0] = __builtin_bit_cast(u32x4, x);
    } else {
        f16v8 x;
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = (_Float16)v[j];
        f.w[0] = __builtin_bit_cast(u32x4, x);
    }
    return f;
}

// acc (32 x 32) += A (32 x 16) B (16 x 32).  Lane l holds row l % 32 of A and
// column l % 32 of B, steps 8 (l / 32) .. + 7; it holds column l % 32 of acc
// and its rows 8 (r / 4) + 4 (l / 32) + r % 4.  fp32 runs eight products of
// two steps each: both operands name the steps in the same order.
template <typename T>
__device__ __forceinline__ void mma(f32x16 &acc, const Frag<T> &a, const Frag<T> &b) {
    if constexpr (T::bytes == 4) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            acc = __builtin_amdgcn_mfma_f32_32x32x2f32(frag_get<T>(a, j), frag_get<T>(b, j), acc, 0,
                                                       0, 0);
    } else if constexpr (__is_same(T, BF16)) {
        acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16v8, a.w[0]),
                                                      __builtin_bit_cast(bf16v8, b.w[0]), acc, 0, 0, 0);
    } else {
        acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16v8, a.w[0]),
                                                     __builtin_bit_cast(f16v8, b.w[0]), acc, 0, 0, 0);
    }
}

// Row of a 32-row tile that row m of the A operand carries, chosen so that a
// lane's results r = 8 t + j are rows 16 t + 8 (lane / 32) + j of the tile:
// eight consecutive ones, which is the order in which the next product's B
// operand wants them.  The results feed it without leaving the registers, and
// one generator call covers them.
__device__ __forceinline__ int a_row(int m) {
    return 16 * (m >> 4) + 8 * ((m >> 2) & 1) + 4 * ((m >> 3) & 1) + (m & 3);
}

// Rows row0 .. row0 + ROWS - 1 of a strided tensor into registers, in 16-byte
// chunks over NT threads, zeros outside rows < limit and columns < D; put()
// writes them to LDS rows of PITCH elements.
template <typename T, int DP, int ROWS, int NT, int PITCH>
struct TileCopy {
    typedef typename T::raw_t raw_t;
    static constexpr int EPC = 16 / T::bytes;
    static constexpr int CPR = DP / EPC;
    static constexpr int N = (ROWS * CPR + NT - 1) / NT;
    u32x4 reg[N];

    __device__ __forceinline__ void fetch(const raw_t *base, int64_t stride, int row0, int limit, int D,
                                          bool vec, int t) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int c = t + n * NT, r = c / CPR, col = (c - r * CPR) * EPC;
            u32x4 v = {0, 0, 0, 0};
            if ((ROWS * CPR % NT == 0 || c < ROWS * CPR) && row0 + r < limit && col < D) {
                const raw_t *src = base + (int64_t)(row0 + r) * stride + col;
                if (vec) {
                    v = *(const u32x4 *)src;
                } else {
                    raw_t e[EPC];
#pragma unroll
                    for (int j = 0; j < EPC; ++j) e[j] = col + j < D ? src[j] : raw_t(0);
                    __builtin_memcpy(&v, e, 16);
                }
            }
            reg[n] = v;
        }
    }
    __device__ __forceinline__ void put(raw_t *lds, int t) const {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int c = t + n * NT, r = c / CPR, col = (c - r * CPR) * EPC;
            if (ROWS * CPR % NT == 0 || c < ROWS * CPR) *(u32x4 *)(lds + r * PITCH + col) = reg[n];
        }
    }
};

// Eight elements from column col of a global row (zeros at and past D).
template <typename T>
__device__ __forceinline__ Frag<T> frag_global(const typename T::raw_t *row, int col, int D, bool ok,
                                               bool vec) {
    typedef typename T::raw_t raw_t;
    constexpr int EPC = 16 / T::bytes;
    Frag<T> f;
#pragma unroll
    for (int n = 0; n < T::bytes / 2; ++n) {
        u32x4 v = {0, 0, 0, 0};
        const int c = col + n * EPC;
        if (ok && c < D) {
            if (vec) {
                v = *(const u32x4 *)(row + c);
            } else {
                raw_t e[EPC];
#pragma unroll
                for (int j = 0; j < EPC; ++j) e[j] = c + j < D ? row[c + j] : raw_t(0);
                __builtin_memcpy(&v, e, 16);
            }
        }
        f.w[n] = v;
    }
    return f;
}

// Eight elements from an LDS row (16-byte aligned).
template <typename T>
__device__ __forceinline__ Frag<T> frag_lds(const typename T::raw_t *p) {
    Frag<T> f;
#pragma unroll
    for (int n = 0; n < T::bytes / 2; ++n) f.w[n] = *(const u32x4 *)(p + n * (16 / T::bytes));
    return f;
}

// A operand of a transposed tile: lane l gets column col0 + l % 32 of LDS
// rows row0 + 8 (l / 32) .. + 7.  A lane reads each element on its own.
template <typename T, int PITCH>
__device__ __forceinline__ Frag<T> frag_lds_transposed(const typename T::raw_t *lds, int row0, int col0,
                                                       int lane) {
    Frag<T> f;
    const typename T::raw_t *p = lds + (row0 + 8 * (lane >> 5)) * PITCH + col0 + (lane & 31);
    if constexpr (T::bytes == 4) {
#pragma unroll
        for (int j = 0; j < 8; ++j) f.w[j >> 2][j & 3] = p[j * PITCH];
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            f.w[0][j] = (uint32_t)p[2 * j * PITCH] | (uint32_t)p[(2 * j + 1) * PITCH] << 16;
    }
    return f;
}

// Four consecutive elements of an output row.
template <typename T>
__device__ __forceinline__ void store4(typename T::raw_t *row, int col, int D, bool vec, float a, float b,
                                       float c, float d) {
    if (col >= D) return;
    const float v[4] = {a, b, c, d};
    if (vec) {
        if constexpr (T::bytes == 4) {
            *(tokens_f32x4 *)(row + col) = tokens_f32x4{a, b, c, d};
        } else {
            u32x2 w;
            w[0] = (uint32_t)to_bits<T>(a) | (uint32_t)to_bits<T>(b) << 16;
            w[1] = (uint32_t)to_bits<T>(c) | (uint32_t)to_bits<T>(d) << 16;
            *(u32x2 *)(row + col) = w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (col + j < D) row[col + j] = to_bits<T>(v[j]);
    }
}

// ----------------------------------------------------- relative positions

// Bucket of one side that distance d >= 0 falls into: the last one whose
// first distance is at most d.
__device__ __forceinline__ int bucket_of(const uint16_t *starts, int side, int d) {
    int lo = 0, hi = side - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (starts[mid] <= d) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// A relative position's place in the distance table: -border .. border
// (bidirectional) or -border .. 0; beyond them the bucket no longer changes.
__device__ __forceinline__ int lut_index(const AttnParams &p, int rel) {
    return min(max(rel + p.border, 0), p.lut - 1);
}

// Fills lut[index] = bias of head h, times log2(e) (the scores are kept in
// base 2), for every place of the distance table.
template <typename T>
__device__ __forceinline__ void fill_lut(const AttnParams &p, int h, float *lut, uint16_t *starts, int t,
                                         int nt) {
    for (int i = t; i < p.side; i += nt) starts[i] = p.starts[i];
    __syncthreads();
    for (int i = t; i < p.lut; i += nt) {
        const int rel = i - p.border;
        int b = bucket_of(starts, p.side, rel < 0 ? -rel : (p.bidirectional ? rel : 0));
        if (p.bidirectional && rel > 0) b += p.side;
        const size_t at = (size_t)b * p.H + h;
        float v;
        if (p.table_f32) v = ((const float *)p.table)[at];
        else v = T::from_raw(((const typename T::raw_t *)p.table)[at]);
        lut[i] = v * kLog2e;
    }
}

// Blocks of one XCD (every eighth of the launch) take consecutive logical
// blocks: the tiles of one head read the same K and V from one L2.
__device__ __forceinline__ int xcd_contiguous_block(int n) {
    const int per = (n + 7) >> 3;
    return (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
}

__device__ __forceinline__ int sequence_length(const AttnParams &p, int b) {
    return p.lengths ? min(max(p.lengths[b], 0), p.Lk) : p.Lk;
}

}  // namespace gs
#endif
